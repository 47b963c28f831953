// Rotary positions, alone and fused into the write of new tokens into a paged
// cache.
//
// Pair i of a head at position t is turned by theta = t * f_i:
//   (a, b) -> m * (a cos(theta) - b sin(theta), a sin(theta) + b cos(theta)).
// The phase is kept as a fraction of a full turn in 64-bit fixed point:
// turn_i = f_i / (2 pi) * 2^64, so that t * turn_i modulo 2^64 -- one wrapping
// integer product -- is the exactly reduced phase at every position, where a
// product in 32-bit floating point is off by 0.03 radians at a million.  Its
// upper 32 bits, read as a signed fraction in [-1/2, 1/2), go to sincospif.
//
// What bounds it: memory, once each element's load and store is 16 bytes wide
// and a thread's angles (the instructions are in sincospif) are shared by all
// heads it handles.
#include "decode_common.cuh"
#include "paged_internal.cuh"

namespace mkv {
namespace {

constexpr int RT = 256;   // threads per block

struct alignas(16) Vec16 {
  uint32_t w[4];
};

template <typename T>
struct Elem;
template <>
struct Elem<__half> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void unpack(const Vec16& v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&v.w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  static __device__ __forceinline__ Vec16 pack(const float (&f)[8]) {
    Vec16 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      v.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return v;
  }
  static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void unpack(const Vec16& v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(v.w[i] << 16);
      f[2 * i + 1] = __uint_as_float(v.w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ Vec16 pack(const float (&f)[8]) {
    Vec16 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      v.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return v;
  }
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Elem<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void unpack(const Vec16& v, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v.w[i]);
  }
  static __device__ __forceinline__ Vec16 pack(const float (&f)[4]) {
    Vec16 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.w[i] = __float_as_uint(f[i]);
    return v;
  }
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};

// m * (cos, sin) of position * turn.
__device__ __forceinline__ void angle(int32_t pos, uint64_t turn, float mult, float sin_mult,
                                      float& c, float& s) {
  const uint64_t phase = (uint64_t)(int64_t)pos * turn;
  const float half_turns = (float)(int32_t)(uint32_t)(phase >> 32) * 4.656612873077393e-10f;  // 2^-31
  sincospif(half_turns, &s, &c);
  c *= mult;
  s *= sin_mult;
}

// Angles of one thread's unit: V pairs (half pairs: two vectors of V elements,
// rot/2 apart) or V/2 pairs (interleaved: one vector).
template <int NP>
__device__ __forceinline__ void angles(const mkv_rope_plan& plan, int first, int32_t pos, float sign,
                                       float (&c)[NP], float (&s)[NP]) {
#pragma unroll
  for (int i = 0; i < NP; ++i) angle(pos, plan.turn[first + i], plan.mult, plan.mult * sign, c[i], s[i]);
}

template <int V>
__device__ __forceinline__ void turn_half(float (&a)[V], float (&b)[V], const float (&c)[V],
                                          const float (&s)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float x = a[i], y = b[i];
    a[i] = x * c[i] - y * s[i];
    b[i] = x * s[i] + y * c[i];
  }
}
template <int V>
__device__ __forceinline__ void turn_inter(float (&a)[V], const float (&c)[V / 2],
                                           const float (&s)[V / 2]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const float x = a[2 * i], y = a[2 * i + 1];
    a[2 * i] = x * c[i] - y * s[i];
    a[2 * i + 1] = x * s[i] + y * c[i];
  }
}

// i / units and i % units of a 64-bit i; nearly always in 32 bits.
__device__ __forceinline__ void split_index(int64_t i, int units, int64_t& q, int& r) {
  if (i < (int64_t)1 << 32) {
    const uint32_t u = (uint32_t)i;
    q = u / (uint32_t)units;
    r = (int)(u - (uint32_t)q * (uint32_t)units);
  } else {
    q = i / units;
    r = (int)(i - q * units);
  }
}

// One unit (first vector at e0; half pairs: second at e1) of HB heads at a time,
// so that their loads are in flight together: rotated where `turns`, else
// copied as it is.  load(h) and store(h, first, second) know the addresses.
template <typename T, bool HALF, typename Load, typename Store>
__device__ __forceinline__ void turn_heads(int h0, int h1, bool turns, const float* c_, const float* s_,
                                           Load load, Store store) {
  using E = Elem<T>;
  constexpr int V = E::V, NP = HALF ? V : V / 2, HB = HALF ? 2 : 4;
  float c[NP], s[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) c[i] = c_[i], s[i] = s_[i];
  for (int h = h0; h < h1; h += HB) {
    Vec16 a[HB], d[HB];
#pragma unroll
    for (int k = 0; k < HB; ++k)
      if (h + k < h1) load(h + k, a[k], d[k]);
#pragma unroll
    for (int k = 0; k < HB; ++k)
      if (h + k < h1) {
        if (turns) {
          float fa[V];
          E::unpack(a[k], fa);
          if constexpr (HALF) {
            float fb[V];
            E::unpack(d[k], fb);
            turn_half<V>(fa, fb, c, s);
            d[k] = E::pack(fb);
          } else {
            turn_inter<V>(fa, c, s);
          }
          a[k] = E::pack(fa);
        }
        store(h + k, a[k], d[k]);
      }
  }
}

// ---------------------------------------------------------------------------
// 16-byte form: a thread takes one unit of one token for `heads_per` heads.
// 4 x 32768 tokens of 8 bf16 heads of 128: 81 us, 6.65 TB/s, 99 % of a copy; fp32,
// 64 of 96 interleaved, 28 heads: 28.5 us, 6.2 TB/s; one step of 8 x 32 heads: 2.1
// us in a graph, a launch.
// grid: (ceil(tokens * units / 256), ceil(heads / heads_per), batch)
// ---------------------------------------------------------------------------
template <typename T, bool HALF>
__global__ void __launch_bounds__(RT) rope_vec_kernel(const __grid_constant__ RopeParams p) {
  griddep_wait();
  griddep_launch();
  constexpr int V = Elem<T>::V, NP = HALF ? V : V / 2;
  int64_t t;
  int u;
  const int64_t idx = (int64_t)blockIdx.x * RT + threadIdx.x;
  split_index(idx, p.units, t, u);
  if (t >= p.tokens) return;
  const int b = blockIdx.z;
  const int h0 = blockIdx.y * p.heads_per, h1 = min(p.heads, h0 + p.heads_per);
  const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + t * p.xs[1];
  T* o = static_cast<T*>(p.out) + b * p.os[0] + t * p.os[1];
  const bool turns = u < p.rot_units;
  float c[NP], s[NP];
  if (turns) {
    const int32_t pos = p.pos ? p.pos[b * p.pos_stride + t] : (int32_t)(p.first_pos + t);
    angles<NP>(p.plan, u * NP, pos, p.sign, c, s);
  }
  const int e0 = turns ? u * V : p.plan.rot_dim + (u - p.rot_units) * V, e1 = e0 + p.plan.rot_dim / 2;
  const int64_t xh = p.xs[2], oh = p.os[2];
  turn_heads<T, HALF>(
      h0, h1, turns, c, s,
      [&](int h, Vec16& a, Vec16& d) {
        a = *reinterpret_cast<const Vec16*>(x + h * xh + e0);
        if (HALF && turns) d = *reinterpret_cast<const Vec16*>(x + h * xh + e1);
      },
      [&](int h, const Vec16& a, const Vec16& d) {
        *reinterpret_cast<Vec16*>(o + h * oh + e0) = a;
        if (HALF && turns) *reinterpret_cast<Vec16*>(o + h * oh + e1) = d;
      });
}

// Element form for sizes, strides or addresses that 16-byte accesses do not
// fit: a unit is one pair, or one copied element.  Its 2-byte accesses, one head at
// a time, bound it: 4 x 32768 tokens of 8 fp16 heads of 128 off a 16-byte boundary
// take 169 us, 3.2 TB/s (80 us on one); heads of 80 with 40 in half pairs 179 us,
// 1.9 TB/s (all 80: 54).
template <typename T>
__global__ void __launch_bounds__(RT) rope_elem_kernel(const __grid_constant__ RopeParams p) {
  griddep_wait();
  griddep_launch();
  using E = Elem<T>;
  int64_t t;
  int u;
  split_index((int64_t)blockIdx.x * RT + threadIdx.x, p.units, t, u);
  if (t >= p.tokens) return;
  const int b = blockIdx.z;
  const int h0 = blockIdx.y * p.heads_per, h1 = min(p.heads, h0 + p.heads_per);
  const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + t * p.xs[1];
  T* o = static_cast<T*>(p.out) + b * p.os[0] + t * p.os[1];
  if (u >= p.rot_units) {
    const int e = p.plan.rot_dim + (u - p.rot_units);
    for (int h = h0; h < h1; ++h) o[h * p.os[2] + e] = x[h * p.xs[2] + e];
    return;
  }
  const int32_t pos = p.pos ? p.pos[b * p.pos_stride + t] : (int32_t)(p.first_pos + t);
  float c, s;
  angle(pos, p.plan.turn[u], p.plan.mult, p.plan.mult * p.sign, c, s);
  const int e0 = p.plan.interleaved ? 2 * u : u;
  const int e1 = p.plan.interleaved ? 2 * u + 1 : u + p.plan.rot_dim / 2;
  for (int h = h0; h < h1; ++h) {
    const float a = E::get(x[h * p.xs[2] + e0]), d = E::get(x[h * p.xs[2] + e1]);
    o[h * p.os[2] + e0] = E::put(a * c - d * s);
    o[h * p.os[2] + e1] = E::put(a * s + d * c);
  }
}

template <typename T>
cudaError_t launch_rope_t(const RopeParams& p, bool vec, cudaStream_t st) {
  const int64_t blocks = (p.tokens * p.units + RT - 1) / RT;
  const dim3 grid((unsigned)blocks, (p.heads + p.heads_per - 1) / p.heads_per, p.batch);
  if (!vec) return launch_kernel(rope_elem_kernel<T>, grid, dim3(RT), 0, st, true, 0, p);
  if (p.plan.interleaved) return launch_kernel(rope_vec_kernel<T, false>, grid, dim3(RT), 0, st, true, 0, p);
  return launch_kernel(rope_vec_kernel<T, true>, grid, dim3(RT), 0, st, true, 0, p);
}

// ---------------------------------------------------------------------------
// append: rows of new tokens into their pages.  The heads of a token are one
// list: keys, values, queries; a thread takes one unit of one token for
// `heads_per` entries of the list.  32182 tokens of 8 KV and 32 query heads of
// 128, bf16 into e4m3: 123 us, 5.9 TB/s; a step of 8 tokens: 2.9 us in a graph.
// grid: (ceil(n * units / 256), ceil(heads_total / heads_per))
// ---------------------------------------------------------------------------
// Eight elements from e on of a cache row; E4M3: times `inv`, saturated.
template <typename T, bool E4M3>
__device__ __forceinline__ void store_row_f32(uint8_t* row, int e, const float (&f)[8], float inv) {
  if constexpr (E4M3) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] * inv, f[4 * i + 1] * inv),
                                                   __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv),
                                                   __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2*>(row + e) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<Vec16*>(row + 2 * e) = Elem<T>::pack(f);
  }
}
template <typename T, bool E4M3>
__device__ __forceinline__ void store_row(uint8_t* row, int e, const Vec16& v, float inv) {
  if constexpr (E4M3) {
    float f[8];
    Elem<T>::unpack(v, f);
    store_row_f32<T, true>(row, e, f, inv);
  } else {
    *reinterpret_cast<Vec16*>(row + 2 * e) = v;
  }
}

template <typename T, bool HALF, bool E4M3>
__global__ void __launch_bounds__(RT) append_rows_kernel(const __grid_constant__ AppendRowsParams p) {
  griddep_wait();
  griddep_launch();
  using E = Elem<T>;
  constexpr int V = 8, NP = HALF ? V : V / 2, HB = 2;
  int64_t t;
  int u;
  split_index((int64_t)blockIdx.x * RT + threadIdx.x, p.units, t, u);
  if (t >= p.a.n) return;
  const int H = p.c.n_kv_heads, ps = p.c.page_size;
  const int l0 = blockIdx.y * p.heads_per, l1 = min(p.heads_total, l0 + p.heads_per);
  const int32_t slot = p.a.slot[t];
  const int32_t pos = p.a.pos ? p.a.pos[t] : slot;
  int64_t seq = t;
  int32_t page = -1;
  bool live = false;
  if (l0 < 2 * H && slot >= 0) {
    if (p.a.seq) seq = p.a.seq[t];
    live = seq >= 0 && seq < p.c.batch && slot / ps < p.c.max_pages &&
           !((p.a.acc || p.a.pos_meta) && slot >= p.a.meta_stride);
    if (live) {
      page = p.c.page_table[seq * p.c.table_stride + slot / ps];
      live = page >= 0 && page < p.c.n_pages;
    }
    if (!live && p.c.status && u == 0) atomicOr(p.c.status, DEV_ERR_CHECK);
  }
  const int rot = p.plan.rot_dim;
  const bool turns = u < p.rot_units, two = HALF && turns;
  float c[NP], s[NP];
  if (turns) angles<NP>(p.plan, u * NP, pos, 1.f, c, s);
  // elements of the unit: one vector, or two half a rotation apart
  const int e0 = turns ? u * V : rot + (u - p.rot_units) * V, e1 = e0 + rot / 2;
  if (live) {
    const int row_bytes = p.c.head_dim * (E4M3 ? 1 : 2);
    const int64_t row0 = ((int64_t)page * H * ps + slot % ps) * row_bytes, head_bytes = (int64_t)ps * row_bytes;
    // keys: rotated in fp32 and rounded once, to the cache's type
    const T* x = static_cast<const T*>(p.a.k) + t * p.a.k_stride[0];
    const int64_t xh = p.a.k_stride[1];
    uint8_t* pool = static_cast<uint8_t*>(p.c.k_pages) + row0;
    const float* scales = E4M3 ? p.c.k_scale : nullptr;
    for (int h = l0; h < min(l1, H); h += HB) {
      Vec16 a[HB], d[HB];
#pragma unroll
      for (int k = 0; k < HB; ++k)
        if (h + k < min(l1, H)) {
          a[k] = *reinterpret_cast<const Vec16*>(x + (h + k) * xh + e0);
          if (two) d[k] = *reinterpret_cast<const Vec16*>(x + (h + k) * xh + e1);
        }
#pragma unroll
      for (int k = 0; k < HB; ++k)
        if (h + k < min(l1, H)) {
          uint8_t* row = pool + (h + k) * head_bytes;
          const float inv = scales ? 1.f / scales[h + k] : 1.f;
          if (turns) {
            float fa[V], fb[V];
            E::unpack(a[k], fa);
            if constexpr (HALF) {
              E::unpack(d[k], fb);
              turn_half<V>(fa, fb, c, s);
              store_row_f32<T, E4M3>(row, e1, fb, inv);
            } else {
              turn_inter<V>(fa, c, s);
            }
            store_row_f32<T, E4M3>(row, e0, fa, inv);
          } else {
            store_row<T, E4M3>(row, e0, a[k], inv);
          }
          if (u == 0) {
            const int64_t m = (seq * H + h + k) * p.a.meta_stride + slot;
            if (p.a.acc) p.a.acc[m] = 0.f;
            if (p.a.pos_meta) p.a.pos_meta[m] = pos;
          }
        }
    }
    // values
    const T* y = static_cast<const T*>(p.a.v) + t * p.a.v_stride[0];
    const int64_t yh = p.a.v_stride[1];
    uint8_t* vpool = static_cast<uint8_t*>(p.c.v_pages) + row0;
    const float* vscales = E4M3 ? p.c.v_scale : nullptr;
    const int v0 = max(l0 - H, 0), v1 = min(l1 - H, H);
    for (int h = v0; h < v1; h += HB) {
      Vec16 a[HB], d[HB];
#pragma unroll
      for (int k = 0; k < HB; ++k)
        if (h + k < v1) {
          a[k] = *reinterpret_cast<const Vec16*>(y + (h + k) * yh + e0);
          if (two) d[k] = *reinterpret_cast<const Vec16*>(y + (h + k) * yh + e1);
        }
#pragma unroll
      for (int k = 0; k < HB; ++k)
        if (h + k < v1) {
          uint8_t* row = vpool + (h + k) * head_bytes;
          const float inv = vscales ? 1.f / vscales[h + k] : 1.f;
          store_row<T, E4M3>(row, e0, a[k], inv);
          if (two) store_row<T, E4M3>(row, e1, d[k], inv);
        }
    }
  }
  if (l1 > 2 * H) {
    const T* x = static_cast<const T*>(p.a.q) + t * p.a.q_stride[0];
    T* o = static_cast<T*>(p.a.q_out) + t * p.a.q_out_stride[0];
    const int64_t xh = p.a.q_stride[1], oh = p.a.q_out_stride[1];
    turn_heads<T, HALF>(
        max(l0 - 2 * H, 0), l1 - 2 * H, turns, c, s,
        [&](int h, Vec16& a, Vec16& d) {
          a = *reinterpret_cast<const Vec16*>(x + h * xh + e0);
          if (two) d = *reinterpret_cast<const Vec16*>(x + h * xh + e1);
        },
        [&](int h, const Vec16& a, const Vec16& d) {
          *reinterpret_cast<Vec16*>(o + h * oh + e0) = a;
          if (two) *reinterpret_cast<Vec16*>(o + h * oh + e1) = d;
        });
  }
}

template <typename T, bool E4M3>
cudaError_t launch_append_t(const AppendRowsParams& p, cudaStream_t st) {
  const int64_t blocks = (p.a.n * p.units + RT - 1) / RT;
  const dim3 grid((unsigned)blocks, (p.heads_total + p.heads_per - 1) / p.heads_per);
  if (p.plan.interleaved || p.rot_units == 0)
    return launch_kernel(append_rows_kernel<T, false, E4M3>, grid, dim3(RT), 0, st, true, 0, p);
  return launch_kernel(append_rows_kernel<T, true, E4M3>, grid, dim3(RT), 0, st, true, 0, p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, bool vec, cudaStream_t st) {
  switch (dtype) {
    case MKV_DT_F16: return launch_rope_t<__half>(p, vec, st);
    case MKV_DT_BF16: return launch_rope_t<__nv_bfloat16>(p, vec, st);
    default: return launch_rope_t<float>(p, vec, st);
  }
}

cudaError_t launch_append_rows(const AppendRowsParams& p, cudaStream_t st) {
  const bool e4m3 = p.c.dtype == MKV_DT_E4M3;
  if (p.a.in_dtype == MKV_DT_F16)
    return e4m3 ? launch_append_t<__half, true>(p, st) : launch_append_t<__half, false>(p, st);
  return e4m3 ? launch_append_t<__nv_bfloat16, true>(p, st) : launch_append_t<__nv_bfloat16, false>(p, st);
}

}  // namespace mkv
