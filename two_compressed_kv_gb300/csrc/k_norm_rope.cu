// RMS norms of query and key heads and their rotation in one pass, and the
// gradients.
//
//   n = x r,  r = 1 / sqrt(mean(x^2) + eps),  y = R(pos) (n w)
//   u = R(pos)^T dy,  e = u w:  dx = r (e - n mean(e n)),  dw = sum of u n
//
// A group of 1 to 32 lanes takes one token's heads one after another; a lane holds
// the same unit (two vectors half a rotation apart, or one vector, or one pair) of
// each of them, so that its angles and weights serve all heads, and sums over a
// head are a few shuffles.  Every element is read once and written by the lane
// that read it.
//
// What bounds it: memory, as long as enough loads are in flight beside the sums over a
// head: two heads at a time, the next two loaded while these are worked on.  8192 x 4
// tokens of 32 + 8 bf16 heads of 128: 128 us, 5.2 TB/s; the gradient of 4099 x 4 tokens
// of 16 + 16: 82 us, 4.9 TB/s; 8 tokens: 3.9 us.  (One head at a time, not ahead: 168
// and 172 us; more resident warps with fewer registers: 162 to 185; four heads: 134.)
#include <type_traits>

#include "decode_common.cuh"
#include "paged_internal.cuh"
#include "rope_common.cuh"

namespace mkv {
namespace {

constexpr int NT = 256;   // threads per block

enum { ELEM = 0, HALF = 1, INTER = 2 };

// A unit of one head: E elements in registers.
// A vector of W 32-bit words and its values, two at a time.
template <int W>
struct alignas(4 * W) Words {
  uint32_t w[W];
};
__device__ __forceinline__ float2 two_of(const uint32_t* w, int i, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(w + i));
}
__device__ __forceinline__ float2 two_of(const uint32_t* w, int i, __nv_bfloat16) {
  return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ float2 two_of(const uint32_t* w, int i, float) {
  return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
}
__device__ __forceinline__ void two_to(uint32_t* w, int i, float2 v, __half) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  w[i] = *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void two_to(uint32_t* w, int i, float2 v, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  w[i] = *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void two_to(uint32_t* w, int i, float2 v, float) {
  w[2 * i] = __float_as_uint(v.x);
  w[2 * i + 1] = __float_as_uint(v.y);
}

template <typename T, int FORM, int BYTES>
struct Unit {
  static constexpr int V = FORM == ELEM ? 1 : BYTES / (int)sizeof(T);
  static constexpr int E = FORM == INTER ? V : 2 * V;        // elements
  static constexpr int NP = E / 2;                           // pairs
  struct Raw {                                               // as loaded
    typename std::conditional<FORM == ELEM, T, Words<BYTES / 4>>::type a, b;
  };
  int e0, e1;      // first element of the unit, and of its second half (ELEM, HALF)
  bool there;      // the head has this unit
  bool turns;      // rotated, else copied (then ELEM and HALF have a first half only)
  __device__ __forceinline__ Unit(const mkv_rope_plan& plan, int u, int units, int rot_units) {
    there = u < units;
    turns = u < rot_units;
    const int rot = plan.rot_dim;
    if (!turns) {
      e0 = there ? rot + (u - rot_units) * V : 0;
      e1 = e0;
    } else if (FORM == ELEM && plan.interleaved) {
      e0 = 2 * u;
      e1 = e0 + 1;
    } else {
      e0 = u * V;
      e1 = FORM == INTER ? e0 : e0 + rot / 2;
    }
  }
  __device__ __forceinline__ Raw load(const T* row, bool live) const {
    Raw r{};
    if (live && there) {
      r.a = *reinterpret_cast<const decltype(r.a)*>(row + e0);
      if (FORM != INTER && turns) r.b = *reinterpret_cast<const decltype(r.b)*>(row + e1);
    }
    return r;
  }
  __device__ __forceinline__ void unpack(const Raw& r, float2 (&f)[NP]) const {
    if constexpr (FORM == ELEM) {
      f[0] = make_float2(Elem<T>::get(r.a), Elem<T>::get(r.b));
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        f[i] = two_of(r.a.w, i, T());
        if (FORM == HALF) f[V / 2 + i] = two_of(r.b.w, i, T());
      }
    }
  }
  __device__ __forceinline__ void store(T* row, const float2 (&f)[NP]) const {
    if constexpr (FORM == ELEM) {
      row[e0] = Elem<T>::put(f[0].x);
      if (turns) row[e1] = Elem<T>::put(f[0].y);
    } else {
      Words<BYTES / 4> x;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) two_to(x.w, i, f[i], T());
      *reinterpret_cast<Words<BYTES / 4>*>(row + e0) = x;
      if (FORM == HALF && turns) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) two_to(x.w, i, f[V / 2 + i], T());
        *reinterpret_cast<Words<BYTES / 4>*>(row + e1) = x;
      }
    }
  }
  // element of the head that value i (of E) is; -1: none
  __device__ __forceinline__ int element(int i) const {
    if (!there) return -1;
    if constexpr (FORM == INTER) return e0 + i;
    return i < V ? e0 + i : turns ? e1 + i - V : -1;
  }
  // the other element of the pair that each value of f[i] is in
  static __device__ __forceinline__ float2 other(const float2 (&f)[NP], int i) {
    if constexpr (FORM == HALF) return f[(i + V / 2) % NP];
    return make_float2(f[i].y, f[i].x);
  }
  // pair that value i belongs to, and whether it is the pair's second element
  static __device__ __forceinline__ int pair_of(int i) { return FORM == HALF ? i % V : i / 2; }
  static __device__ __forceinline__ bool second(int i) { return FORM == HALF ? i >= V : i % 2; }
};

template <typename T>
__device__ __forceinline__ float weight_at(const NormRopeParams& p, int side, int e) {
  if (!p.weight[side]) return 1.f;
  return (p.weight_f32[side] ? static_cast<const float*>(p.weight[side])[e]
                             : Elem<T>::get(static_cast<const T*>(p.weight[side])[e])) + p.offset;
}

// NU: units of a lane; HB: heads whose loads are in flight together.  Grid: blocks of
// the queries, then blocks of the keys; the groups of lanes of a side's blocks walk over
// its items (a token and `heads_per` of its heads) with their units' weights and
// (gradient) sums in registers.  A token's angles and weights come together in two
// factors of every value: y = r (x A + other(x) B), other(x) its pair's other element.
template <typename T, int FORM, int BYTES, int NU, int HB, bool GRAD>
__global__ void __launch_bounds__(NT, FORM == ELEM ? 1 : 2)
    norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  using U = Unit<T, FORM, BYTES>;
  constexpr int E = U::E, NP = U::NP;
  __shared__ uint64_t speeds[MKV_ROPE_MAX_PAIRS];
  __shared__ uint8_t axes[MKV_ROPE_MAX_PAIRS];
  __shared__ float weights[2 * MKV_ROPE_MAX_PAIRS];
  const int lane = threadIdx.x & (p.lanes - 1);
  const int side = blockIdx.x >= p.blocks[0];
  const int block = side ? blockIdx.x - p.blocks[0] : blockIdx.x;
  const int per_block = NT / p.lanes;
  const int64_t groups = (int64_t)p.blocks[side] * per_block;
  const int64_t group = (int64_t)block * per_block + threadIdx.x / p.lanes;
  for (int i = threadIdx.x; i < MKV_ROPE_MAX_PAIRS; i += NT) {
    speeds[i] = p.plan.turn[i];
    axes[i] = p.axes.axis[i];
  }
  griddep_wait();
  griddep_launch();
  for (int i = threadIdx.x; i < p.plan.head_dim; i += NT) weights[i] = weight_at<T>(p, side, i);
  __syncthreads();
  // weights of a lane's values (forward: read again for every token, registers are short)
  auto weight = [&](const U& unit, int i) {
    const int e = unit.element(2 * i), f = unit.element(2 * i + 1);
    return make_float2(e >= 0 ? weights[e] : 0.f, f >= 0 ? weights[f] : 0.f);
  };
  float2 w[GRAD ? NU : 1][NP], dw[GRAD ? NU : 1][NP];
  if constexpr (GRAD) {
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      const U unit(p.plan, lane + n * p.lanes, p.units, p.rot_units);
#pragma unroll
      for (int i = 0; i < NP; ++i) w[n][i] = weight(unit, i), dw[n][i] = make_float2(0.f, 0.f);
    }
  }
  const float share = 1.f / (float)p.plan.head_dim;
  const int heads = p.heads[side], steps = min(p.heads_per, heads);
  const int64_t xh = p.xs[side][2], gh = p.gs[side][2], oh = p.os[side][2];
  // every lane of a warp takes the same number of turns: the shuffles need all of them
  for (int64_t first = 0; first < p.items[side]; first += groups) {
    const int64_t item = first + group;
    const bool there = item < p.items[side];
    int64_t row;
    int chunk;
    split_index(there ? item : 0, p.chunks[side], row, chunk);
    const int64_t b = div_small(row, p.tokens), t = row - b * p.tokens;
    const int h0 = chunk * p.heads_per, h1 = there ? min(heads, h0 + p.heads_per) : h0;
    const T* x = static_cast<const T*>(p.x[side]) + b * p.xs[side][0] + t * p.xs[side][1];
    const T* g = GRAD ? static_cast<const T*>(p.grad[side]) + b * p.gs[side][0] + t * p.gs[side][1] : nullptr;
    T* o = static_cast<T*>(p.out[side]) + b * p.os[side][0] + t * p.os[side][1];
    // the next heads' loads are in flight while these are worked on, the first ones' during
    // the angles
    typename U::Raw rx[HB][NU], rg[GRAD ? HB : 1][NU];
    x += h0 * xh;
    o += h0 * oh;
    if constexpr (GRAD) g += h0 * gh;
    auto load = [&](int h) {
#pragma unroll
      for (int k = 0; k < HB; ++k)
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          const U unit(p.plan, lane + n * p.lanes, p.units, p.rot_units);
          rx[k][n] = unit.load(x + k * xh, h + k < h1);
          if constexpr (GRAD) rg[k][n] = unit.load(g + k * gh, h + k < h1);
        }
      x += HB * xh;
      if constexpr (GRAD) g += HB * gh;
    };
    load(h0);
    float2 A[NU][NP], B[NU][NP];
    {
      int32_t at[MKV_ROPE_MAX_AXES] = {(int32_t)(p.first_pos + t), 0, 0, 0};
      if (p.pos) {
        const int32_t* pos = p.pos + b * p.pos_stride + t;
        at[0] = pos[0];
#pragma unroll
        for (int a = 1; a < MKV_ROPE_MAX_AXES; ++a)
          if (a < p.axes.n_axes) at[a] = pos[a * p.pos_axis_stride];
      }
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        const U unit(p.plan, lane + n * p.lanes, p.units, p.rot_units);
        float c[NP], s[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          c[i] = 1.f, s[i] = 0.f;
          if (unit.turns) {
            const int pair = (lane + n * p.lanes) * NP + i, a = axes[pair];
            const int32_t own = a == 0 ? at[0] : a == 1 ? at[1] : a == 2 ? at[2] : at[3];
            angle(own, speeds[pair], p.plan.mult, p.plan.mult, c[i], s[i]);
          }
        }
        float2 v[NP];
        if constexpr (!GRAD) {
#pragma unroll
          for (int i = 0; i < NP; ++i) v[i] = weight(unit, i);
        }
        // forward: A = w c, B = the other's w times -s or s; back: A = c, B = s or -s
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int e = 2 * i, f = 2 * i + 1, pe = U::pair_of(e), pf = U::pair_of(f);
          A[n][i] = make_float2(c[pe], c[pf]);
          B[n][i] = make_float2(U::second(e) ? s[pe] : -s[pe], U::second(f) ? s[pf] : -s[pf]);
          if constexpr (GRAD) {
            B[n][i] = make_float2(-B[n][i].x, -B[n][i].y);
          } else {
            A[n][i] = mul2(A[n][i], v[i]);
            B[n][i] = mul2(B[n][i], U::other(v, i));
          }
        }
      }
    }
    for (int h = h0; h < h0 + steps; h += HB) {
      float2 f[HB][NU][NP], d[GRAD ? HB : 1][NU][NP];
      float ss[HB], en[HB];
#pragma unroll
      for (int k = 0; k < HB; ++k)
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          const U unit(p.plan, lane + n * p.lanes, p.units, p.rot_units);
          unit.unpack(rx[k][n], f[k][n]);
          if constexpr (GRAD) unit.unpack(rg[k][n], d[k][n]);
        }
      if (h + HB < h0 + steps) load(h + HB);
#pragma unroll
      for (int k = 0; k < HB; ++k) {
        float2 sq = make_float2(0.f, 0.f), along = make_float2(0.f, 0.f);
#pragma unroll
        for (int n = 0; n < NU; ++n) {
#pragma unroll
          for (int i = 0; i < NP; ++i) sq = fma2(f[k][n][i], f[k][n][i], sq);
          if constexpr (GRAD) {
            // u, and the sum of u w x: r times that is the sum of e n
            float2 u[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              u[i] = fma2(U::other(d[k][n], i), B[n][i], mul2(d[k][n][i], A[n][i]));
              along = fma2(mul2(u[i], w[n][i]), f[k][n][i], along);
            }
#pragma unroll
            for (int i = 0; i < NP; ++i) d[k][n][i] = u[i];
          }
        }
        ss[k] = sq.x + sq.y;
        en[k] = along.x + along.y;
      }
      for (int m = p.lanes >> 1; m; m >>= 1)
#pragma unroll
        for (int k = 0; k < HB; ++k) {
          ss[k] += __shfl_xor_sync(~0u, ss[k], m);
          if constexpr (GRAD) en[k] += __shfl_xor_sync(~0u, en[k], m);
        }
#pragma unroll
      for (int k = 0; k < HB; ++k) {
        // absent heads are zeros, which r must not turn into NaN
        const float r = GRAD && h + k >= h1 ? 0.f : rsqrtf(fmaf(ss[k], share, p.eps));
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          const U unit(p.plan, lane + n * p.lanes, p.units, p.rot_units);
          float2 y[NP];
          if constexpr (!GRAD) {
#pragma unroll
            for (int i = 0; i < NP; ++i)
              y[i] = mul2(fma2(U::other(f[k][n], i), B[n][i], mul2(f[k][n][i], A[n][i])), twice(r));
          } else {
            const float mean = en[k] * share * r * r;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
              const float2 u = mul2(d[k][n][i], twice(r));
              dw[n][i] = fma2(u, f[k][n][i], dw[n][i]);
              y[i] = fma2(f[k][n][i], twice(-mean * r), mul2(u, w[n][i]));
            }
          }
          if (h + k < h1 && unit.there) unit.store(o + k * oh, y);
        }
      }
      o += HB * oh;
    }
  }
  if constexpr (GRAD) {
    if (!p.part) return;
    // the block's groups, in their order: [group][head_dim] in shared memory
    extern __shared__ float sums[];
    const int D = p.plan.head_dim;
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      const U unit(p.plan, lane + n * p.lanes, p.units, p.rot_units);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int e = unit.element(i);
        if (e >= 0) sums[(threadIdx.x / p.lanes) * D + e] = i % 2 ? dw[n][i / 2].y : dw[n][i / 2].x;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += NT) {
      float a = 0.f;
      for (int k = 0; k < per_block; ++k) a += sums[k * D + e];
      p.part[(int64_t)blockIdx.x * D + e] = a;
    }
  }
}

// The sums of a side's blocks, in a fixed order: 32 elements a block, 32 warps each a
// thirty-second of the blocks, then the warps'.  grid: (ceil(D / 32), 2)
__global__ void __launch_bounds__(1024) norm_weight_kernel(const __grid_constant__ NormRopeParams p) {
  __shared__ float sm[32][33];
  griddep_wait();
  griddep_launch();
  const int side = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = p.plan.head_dim;
  float* out = p.weight_grad[side];
  if (!out) return;
  const int e = blockIdx.x * 32 + lane;
  const float* part = p.part + (side ? (int64_t)p.blocks[0] * D : 0);
  float a = 0.f;
  if (e < D)
    for (int k = warp; k < p.blocks[side]; k += 32) a += part[(int64_t)k * D + e];
  sm[warp][lane] = a;
  __syncthreads();
  float v = sm[lane][warp];
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  const int to = blockIdx.x * 32 + warp;
  if (lane == 0 && to < D) out[to] = v;
}

template <typename T, int FORM, int BYTES, int NU, int HB, bool GRAD>
cudaError_t launch_form(const NormRopeParams& p, cudaStream_t st) {
  // at most 16 elements a lane and unit pair: 16 KB
  const size_t smem = GRAD && p.part ? (size_t)(NT / p.lanes) * p.plan.head_dim * 4 : 0;
  cudaError_t e = launch_kernel(norm_rope_kernel<T, FORM, BYTES, NU, HB, GRAD>, dim3(p.blocks[0] + p.blocks[1]), dim3(NT),
                                smem, st, true, 0, p);
  if (e != cudaSuccess || !GRAD || !p.part) return e;
  return launch_kernel(norm_weight_kernel, dim3((p.plan.head_dim + 31) / 32, 2), dim3(1024), 0, st, true, 0, p);
}

template <typename T, bool GRAD>
cudaError_t launch_t(const NormRopeParams& p, int form, cudaStream_t st) {
  constexpr int BYTES = norm_vector_bytes(sizeof(T) == 2, GRAD);
  if (form == ELEM) return launch_form<T, ELEM, 4, 8, 1, GRAD>(p, st);
  if (p.units > p.lanes)
    return form == HALF ? launch_form<T, HALF, BYTES, 2, 1, GRAD>(p, st) : launch_form<T, INTER, BYTES, 2, 1, GRAD>(p, st);
  return form == HALF ? launch_form<T, HALF, BYTES, 1, 2, GRAD>(p, st) : launch_form<T, INTER, BYTES, 1, 2, GRAD>(p, st);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int dtype, int form, bool grad, cudaStream_t st) {
  switch (dtype) {
    case MKV_DT_F16: return grad ? launch_t<__half, true>(p, form, st) : launch_t<__half, false>(p, form, st);
    case MKV_DT_BF16: return grad ? launch_t<__nv_bfloat16, true>(p, form, st) : launch_t<__nv_bfloat16, false>(p, form, st);
    default: return grad ? launch_t<float, true>(p, form, st) : launch_t<float, false>(p, form, st);
  }
}

}  // namespace mkv
