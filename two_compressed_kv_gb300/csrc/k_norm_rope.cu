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
// What bounds it: memory.
#include "decode_common.cuh"
#include "paged_internal.cuh"
#include "rope_common.cuh"

namespace mkv {
namespace {

constexpr int NT = 256;   // threads per block

enum { ELEM = 0, HALF = 1, INTER = 2 };

// A unit of one head: E elements in registers.
template <typename T, int FORM>
struct Unit {
  static constexpr int V = FORM == ELEM ? 1 : Elem<T>::V;
  static constexpr int E = FORM == INTER ? V : 2 * V;        // elements
  static constexpr int NP = E / 2;                           // pairs
  int e0, e1;      // first element of the unit, and of its second half (ELEM, HALF)
  bool turns;      // rotated, else copied (then ELEM and HALF have a first half only)
  __device__ __forceinline__ Unit(const mkv_rope_plan& plan, int u, int rot_units) {
    turns = u < rot_units;
    const int rot = plan.rot_dim;
    if (!turns) {
      e0 = rot + (u - rot_units) * V;
      e1 = e0;
    } else if (FORM == ELEM && plan.interleaved) {
      e0 = 2 * u;
      e1 = e0 + 1;
    } else {
      e0 = u * V;
      e1 = e0 + rot / 2;
    }
  }
  __device__ __forceinline__ void load(const T* row, float (&f)[E]) const {
    if constexpr (FORM == ELEM) {
      f[0] = Elem<T>::get(row[e0]);
      f[1] = turns ? Elem<T>::get(row[e1]) : 0.f;
    } else {
      float a[V];
      Elem<T>::unpack(*reinterpret_cast<const Vec16*>(row + e0), a);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = a[i];
      if constexpr (FORM == HALF) {
        Vec16 v{};
        if (turns) v = *reinterpret_cast<const Vec16*>(row + e1);
        Elem<T>::unpack(v, a);
#pragma unroll
        for (int i = 0; i < V; ++i) f[V + i] = a[i];
      }
    }
  }
  __device__ __forceinline__ void store(T* row, const float (&f)[E]) const {
    if constexpr (FORM == ELEM) {
      row[e0] = Elem<T>::put(f[0]);
      if (turns) row[e1] = Elem<T>::put(f[1]);
    } else {
      float a[V];
#pragma unroll
      for (int i = 0; i < V; ++i) a[i] = f[i];
      *reinterpret_cast<Vec16*>(row + e0) = Elem<T>::pack(a);
      if constexpr (FORM == HALF) {
        if (turns) {
#pragma unroll
          for (int i = 0; i < V; ++i) a[i] = f[V + i];
          *reinterpret_cast<Vec16*>(row + e1) = Elem<T>::pack(a);
        }
      }
    }
  }
  // element of the head that f[i] is; -1: none
  __device__ __forceinline__ int element(int i) const {
    if constexpr (FORM == INTER) return e0 + i;
    return i < V ? e0 + i : turns ? e1 + i - V : -1;
  }
  // (cos, sin) of the unit's pairs; sign -1: the transposed rotation
  __device__ __forceinline__ void turn(float (&f)[E], const float (&c)[NP], const float (&s)[NP], float sign) const {
    if (!turns) return;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      constexpr bool inter = FORM == INTER;
      const int a = inter ? 2 * i : i, b = inter ? 2 * i + 1 : i + V;
      const float x = f[a], y = f[b], si = s[i] * sign;
      f[a] = x * c[i] - y * si;
      f[b] = x * si + y * c[i];
    }
  }
};

__device__ __forceinline__ float sum_lanes(float v, int lanes) {
  for (int o = lanes >> 1; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

template <typename T>
__device__ __forceinline__ float weight_at(const NormRopeParams& p, int side, int e) {
  if (!p.weight[side]) return 1.f;
  return (p.weight_f32[side] ? static_cast<const float*>(p.weight[side])[e]
                             : Elem<T>::get(static_cast<const T*>(p.weight[side])[e])) + p.offset;
}

// NU: units of a lane.  Grid: blocks; the groups of lanes of all blocks walk over
// the items (a token and a chunk of the list of its heads, queries first).
template <typename T, int FORM, int NU, bool GRAD>
__global__ void __launch_bounds__(NT) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  using U = Unit<T, FORM>;
  constexpr int E = U::E, NP = U::NP;
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & (p.lanes - 1);
  const int64_t groups = (int64_t)gridDim.x * (NT / p.lanes);
  const int64_t group = (int64_t)blockIdx.x * (NT / p.lanes) + threadIdx.x / p.lanes;
  float dw[GRAD ? 2 : 1][NU][E];
  if constexpr (GRAD) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int n = 0; n < NU; ++n)
#pragma unroll
        for (int i = 0; i < E; ++i) dw[k][n][i] = 0.f;
  }
  // every lane of a warp takes the same number of turns: the shuffles need all of them
  const int64_t rounds = (p.items + groups - 1) / groups;
  for (int64_t round = 0; round < rounds; ++round) {
    const int64_t item = round * groups + group;
    const bool there = item < p.items;
    int64_t row, t;
    int chunk, b;
    split_index(there ? item : 0, p.chunks, row, chunk);
    {
      const int64_t q = div_small(row, p.tokens);
      t = row - q * p.tokens;
      b = (int)q;
    }
    float c[NU][NP], s[NU][NP];
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      const int u = lane + n * p.lanes;
      if (u < p.rot_units) {
        if (p.axes.n_axes) {
          axes_angles<NP>(p.plan, p.axes, p.pos + b * p.pos_stride + t, p.pos_axis_stride, u * NP, 1.f, c[n], s[n]);
        } else {
          const int32_t pos = p.pos ? p.pos[b * p.pos_stride + t] : (int32_t)(p.first_pos + t);
          angles<NP>(p.plan, u * NP, pos, 1.f, c[n], s[n]);
        }
      }
    }
    const int h0 = chunk * p.heads_per, h1 = min(p.heads[0] + p.heads[1], h0 + p.heads_per);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int from = side ? max(h0 - p.heads[0], 0) : h0, to = side ? h1 - p.heads[0] : min(h1, p.heads[0]);
      // the lanes of a warp may have different heads: as many turns as the most of them
      int most = there ? max(0, to - from) : 0;
      most = __reduce_max_sync(~0u, most);
      if (most == 0) continue;
      float w[NU][E];
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        const int u = lane + n * p.lanes;
        const U unit(p.plan, u, p.rot_units);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int e = u < p.units ? unit.element(i) : -1;
          w[n][i] = e >= 0 ? weight_at<T>(p, side, e) : 0.f;
        }
      }
      const T* x = static_cast<const T*>(p.x[side]) + b * p.xs[side][0] + t * p.xs[side][1];
      const T* g = GRAD ? static_cast<const T*>(p.grad[side]) + b * p.gs[side][0] + t * p.gs[side][1] : nullptr;
      T* o = static_cast<T*>(p.out[side]) + b * p.os[side][0] + t * p.os[side][1];
      for (int k = 0; k < most; ++k) {
        const int h = from + k;
        const bool live = there && h < to;
        float f[NU][E], d[NU][E];
        float ss = 0.f;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          const int u = lane + n * p.lanes;
          const U unit(p.plan, u, p.rot_units);
#pragma unroll
          for (int i = 0; i < E; ++i) f[n][i] = d[n][i] = 0.f;
          if (live && u < p.units) {
            unit.load(x + h * p.xs[side][2], f[n]);
            if constexpr (GRAD) unit.load(g + h * p.gs[side][2], d[n]);
          }
#pragma unroll
          for (int i = 0; i < E; ++i) ss += f[n][i] * f[n][i];
        }
        ss = sum_lanes(ss, p.lanes);
        const float r = 1.f / sqrtf(ss / (float)p.plan.head_dim + p.eps);
        if constexpr (!GRAD) {
#pragma unroll
          for (int n = 0; n < NU; ++n) {
            const int u = lane + n * p.lanes;
            const U unit(p.plan, u, p.rot_units);
#pragma unroll
            for (int i = 0; i < E; ++i) f[n][i] = f[n][i] * r * w[n][i];
            unit.turn(f[n], c[n], s[n], 1.f);
            if (live && u < p.units) unit.store(o + h * p.os[side][2], f[n]);
          }
        } else {
          float en = 0.f;
#pragma unroll
          for (int n = 0; n < NU; ++n) {
            const U unit(p.plan, lane + n * p.lanes, p.rot_units);
            unit.turn(d[n], c[n], s[n], -1.f);
#pragma unroll
            for (int i = 0; i < E; ++i) {
              if (live) f[n][i] *= r;
              dw[side][n][i] += d[n][i] * f[n][i];
              d[n][i] *= w[n][i];
              en += d[n][i] * f[n][i];
            }
          }
          en = sum_lanes(en, p.lanes) / (float)p.plan.head_dim;
#pragma unroll
          for (int n = 0; n < NU; ++n) {
            const int u = lane + n * p.lanes;
            const U unit(p.plan, u, p.rot_units);
#pragma unroll
            for (int i = 0; i < E; ++i) f[n][i] = r * (d[n][i] - f[n][i] * en);
            if (live && u < p.units) unit.store(o + h * p.os[side][2], f[n]);
          }
        }
      }
    }
  }
  if constexpr (GRAD) {
    if (!p.part) return;
    // the block's groups, in their order: [group][head_dim] in shared memory, a side at a time
    extern __shared__ float sums[];
    const int D = p.plan.head_dim, here = NT / p.lanes;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        const int u = lane + n * p.lanes;
        const U unit(p.plan, u, p.rot_units);
        if (u < p.units) {
#pragma unroll
          for (int i = 0; i < E; ++i) {
            const int e = unit.element(i);
            if (e >= 0) sums[(threadIdx.x / p.lanes) * D + e] = dw[side][n][i];
          }
        }
      }
      __syncthreads();
      for (int e = threadIdx.x; e < D; e += NT) {
        float a = 0.f;
        for (int k = 0; k < here; ++k) a += sums[k * D + e];
        p.part[((int64_t)blockIdx.x * 2 + side) * D + e] = a;
      }
    }
  }
}

// The blocks' sums, in a fixed order: 32 elements a block, 32 warps each a
// thirty-second of the blocks, then the warps'.  grid: (ceil(D / 32), 2)
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float* part, int blocks, int D, float* out0, float* out1) {
  __shared__ float sm[32][33];
  griddep_wait();
  griddep_launch();
  const int side = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* out = side ? out1 : out0;
  if (!out) return;
  const int e = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (e < D)
    for (int k = warp; k < blocks; k += 32) a += part[((int64_t)k * 2 + side) * D + e];
  sm[warp][lane] = a;
  __syncthreads();
  float v = sm[lane][warp];
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  const int to = blockIdx.x * 32 + warp;
  if (lane == 0 && to < D) out[to] = v;
}

template <typename T, int FORM, int NU>
cudaError_t launch_form(const NormRopeParams& p, bool grad, cudaStream_t st) {
  if (!grad) return launch_kernel(norm_rope_kernel<T, FORM, NU, false>, dim3(p.blocks), dim3(NT), 0, st, true, 0, p);
  // at most 16 elements a lane and unit pair: 16 KB
  const size_t smem = p.part ? (size_t)(NT / p.lanes) * p.plan.head_dim * 4 : 0;
  cudaError_t e = launch_kernel(norm_rope_kernel<T, FORM, NU, true>, dim3(p.blocks), dim3(NT), smem, st, true, 0, p);
  if (e != cudaSuccess || !p.part) return e;
  const int D = p.plan.head_dim;
  return launch_kernel(norm_weight_kernel, dim3((D + 31) / 32, 2), dim3(1024), 0, st, true, 0,
                       static_cast<const float*>(p.part), p.blocks, D, p.weight_grad[0], p.weight_grad[1]);
}

template <typename T>
cudaError_t launch_t(const NormRopeParams& p, int form, bool grad, cudaStream_t st) {
  const int per = (p.units + p.lanes - 1) / p.lanes;
  if (form == HALF) return per == 1 ? launch_form<T, HALF, 1>(p, grad, st) : launch_form<T, HALF, 2>(p, grad, st);
  if (form == INTER) return per == 1 ? launch_form<T, INTER, 1>(p, grad, st) : launch_form<T, INTER, 2>(p, grad, st);
  return launch_form<T, ELEM, 8>(p, grad, st);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int dtype, int form, bool grad, cudaStream_t st) {
  switch (dtype) {
    case MKV_DT_F16: return launch_t<__half>(p, form, grad, st);
    case MKV_DT_BF16: return launch_t<__nv_bfloat16>(p, form, grad, st);
    default: return launch_t<float>(p, form, grad, st);
  }
}

}  // namespace mkv
