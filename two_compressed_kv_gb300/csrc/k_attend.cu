// Attention of many queries over keys in tensors or in pages.
//
//   z_ij = score(q_i, k_j) over the keys j that query i sees, o_i = softmax(z_i) v
//
// One warp takes one query of one head and walks over its keys with a running
// maximum and sum; a lane holds D / 32 channels.
#include <math_constants.h>

#include "attend_internal.cuh"
#include "decode_common.cuh"

namespace mkv {
namespace {

template <int N>
__device__ __forceinline__ void load16(const uint16_t* p, bool bf16, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    f[i] = bf16 ? __uint_as_float((uint32_t)p[i] << 16) : __half2float(__ushort_as_half(p[i]));
}
template <int N>
__device__ __forceinline__ void load8(const uint8_t* p, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(p[i], __NV_E4M3);
    f[i] = __half2float(__half(h));
  }
}

template <int D>
__global__ void __launch_bounds__(128) attend_kernel(const __grid_constant__ AttendParams p) {
  griddep_wait();
  griddep_launch();
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= (int64_t)p.B * p.nq * p.Hq) return;
  const int head = (int)(item % p.Hq);
  const int i = (int)(item / p.Hq % p.nq), b = (int)(item / p.Hq / p.nq);
  const int h = head / p.g;
  const int want_k = p.kv_lens ? p.kv_lens[b] : p.nk, want_q = p.q_lens ? p.q_lens[b] : p.nq;
  const int L = max(0, min(want_k, p.nk));
  int m = max(0, min(want_q, p.nq));
  const bool paged = p.table != nullptr;
  if (paged) {
    m = min(m, L);
    if (p.status && head == 0 && i == 0 && lane == 0 && (L != want_k || (p.q_lens && m != want_q)))
      atomicOr(p.status, DEV_ERR_CHECK);
  }
  if (i >= m) return;
  const int base = L - m;
  const uint64_t valid = m >= 64 ? ~0ull : (1ull << m) - 1;
  uint64_t row = 0;
  int place = base + i;
  if (p.tree) {
    row = p.tree[(int64_t)b * p.nq + i] & valid;
    place = base + __popcll(row & ~(1ull << i));
  }
  int lo = 0, hi = L;
  if (!paged && p.causal) hi = min(L, max(place + 1, p.prefix ? p.prefix[b] : 0));
  if (paged && !p.tree) hi = place + 1;
  if (p.window && !p.tree) {
    lo = max(0, place - p.window + 1);
    if (!paged && !p.causal) hi = min(hi, place + p.window);
  }
  const int32_t* docs = p.docs ? p.docs + b * p.docs_stride : nullptr;
  if (docs && place < 0) hi = 0;
  const int32_t doc = docs && place >= 0 ? docs[place] : 0;
  const float slope = p.slopes ? p.slopes[head] : 0.f;
  const bool e4 = paged && p.cache_type == MKV_DT_E4M3;
  const bool kv_bf16 = paged ? p.cache_type == MKV_DT_BF16 : p.bf16;

  float q[N], o[N], kf[N];
  load16<N>(static_cast<const uint16_t*>(p.q) + b * p.qs[0] + i * p.qs[1] + head * p.qs[2] + lane * N, p.bf16, q);
#pragma unroll
  for (int c = 0; c < N; ++c) o[c] = 0.f;
  float top = -CUDART_INF_F, sum = 0.f;
  const float kscale = e4 && p.k_scale ? p.k_scale[h] : 1.f, vscale = e4 && p.v_scale ? p.v_scale[h] : 1.f;
  for (int j = lo; j < hi; ++j) {
    if (docs && docs[j] != doc) continue;
    int at = j;
    if (p.tree) {
      if (j >= base) {
        if (!(row >> (j - base) & 1)) continue;
        at = base + __popcll(p.tree[(int64_t)b * p.nq + j - base] & valid & ~(1ull << (j - base)));
      }
      if (p.window && place - at >= p.window) continue;
    }
    int64_t ko, vo;
    if (paged) {
      const int page = p.table[b * p.table_stride + j / p.page_size];
      if (page < 0 || page >= p.n_pages) {
        if (p.status && lane == 0) atomicOr(p.status, DEV_ERR_CHECK);
        continue;
      }
      ko = vo = (((int64_t)page * p.H + h) * p.page_size + j % p.page_size) * D;
    } else {
      ko = b * p.ks[0] + j * p.ks[1] + h * p.ks[2];
      vo = b * p.vs[0] + j * p.vs[1] + h * p.vs[2];
    }
    if (e4) load8<N>(static_cast<const uint8_t*>(p.k) + ko + lane * N, kf);
    else load16<N>(static_cast<const uint16_t*>(p.k) + ko + lane * N, kv_bf16, kf);
    float z = 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c) z += q[c] * kf[c];
#pragma unroll
    for (int s = 16; s; s >>= 1) z += __shfl_xor_sync(~0u, z, s);
    z *= p.scale * kscale;
    if (p.cap > 0.f) z = p.cap * tanhf(z / p.cap);
    z -= slope * fabsf((float)(place - at));
    if (z > top) {
      const float f = expf(top - z);
      top = z;
      sum *= f;
#pragma unroll
      for (int c = 0; c < N; ++c) o[c] *= f;
    }
    const float w = expf(z - top);
    sum += w;
    if (e4) load8<N>(static_cast<const uint8_t*>(p.v) + vo + lane * N, kf);
    else load16<N>(static_cast<const uint16_t*>(p.v) + vo + lane * N, kv_bf16, kf);
#pragma unroll
    for (int c = 0; c < N; ++c) o[c] += w * kf[c];
  }
  const float inv = sum > 0.f ? vscale / sum : 0.f;
  uint16_t* out = static_cast<uint16_t*>(p.out) + b * p.os[0] + i * p.os[1] + head * p.os[2] + lane * N;
#pragma unroll
  for (int c = 0; c < N; ++c)
    out[c] = p.bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(o[c] * inv)) : __half_as_ushort(__float2half_rn(o[c] * inv));
  if (p.lse && lane == 0) p.lse[((int64_t)b * p.nq + i) * p.Hq + head] = top + logf(sum);
}

}  // namespace

cudaError_t launch_attend(const AttendParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)(((int64_t)p.B * p.nq * p.Hq + 3) / 4)), block(128);
  switch (p.D) {
    case 64: return launch_kernel(attend_kernel<64>, grid, block, 0, st, true, 0, p);
    case 128: return launch_kernel(attend_kernel<128>, grid, block, 0, st, true, 0, p);
    default: return launch_kernel(attend_kernel<256>, grid, block, 0, st, true, 0, p);
  }
}

}  // namespace mkv
