// Vectors of elements and rotated pairs: shared by the rotary kernels.
#pragma once

#include "paged_internal.cuh"

namespace mkv {

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

// The same with several axes: pos points at the token's place of axis 0.
template <int NP>
__device__ __forceinline__ void axes_angles(const mkv_rope_plan& plan, const mkv_rope_axes& axes, const int32_t* pos,
                                            int64_t axis_stride, int first, float sign, float (&c)[NP], float (&s)[NP]) {
  int32_t at[MKV_ROPE_MAX_AXES];
#pragma unroll
  for (int a = 0; a < MKV_ROPE_MAX_AXES; ++a) at[a] = a < axes.n_axes ? pos[a * axis_stride] : 0;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int a = axes.axis[first + i];
    const int32_t own = a == 0 ? at[0] : a == 1 ? at[1] : a == 2 ? at[2] : at[3];
    angle(own, plan.turn[first + i], plan.mult, plan.mult * sign, c[i], s[i]);
  }
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

}  // namespace mkv
