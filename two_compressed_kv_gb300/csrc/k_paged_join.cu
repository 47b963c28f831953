// Second half of the paged attention: the parts of split streams joined, and
// the softmax weights added up for eviction.
#include <math_constants.h>

#include "decode_common.cuh"
#include "paged_internal.cuh"
#include "ptx.cuh"

namespace mkv {
namespace {

constexpr int JT = 256;

// ---------------------------------------------------------------------------
// join: o = sum_k o_k exp2(m_k - M) / sum_k l_k exp2(m_k - M) over the parts k
// of one stream, in a fixed order.  The parts lie in L2; a CTA takes one query
// head, its threads 4 elements each of every (4 T / D)-th part.  T = 1024 threads
// where the heads are so few that all such CTAs run at once: a part from every
// CTA of the split kernel is then still a few loads per thread (one stream of a
// million tokens, 8 heads: 135 us for the whole call with 256 threads, 102 with
// 1024).  Bound by three dependent latencies of L2: lengths, shares, parts.
// grid: streams * g
// ---------------------------------------------------------------------------
template <int D, int T>
__global__ void __launch_bounds__(T) paged_join_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int LD = D / 4, NG = T / LD;       // threads of a part, parts at a time
  __shared__ float4 so[NG][LD];
  __shared__ float sm[NG], sl[NG];
  const int64_t row = blockIdx.x;
  const int64_t stream = row / p.g;
  const int head = (int)(row - stream * p.g);
  const int b = (int)(stream / p.H), h = (int)(stream - (int64_t)b * p.H);
  const int grp = threadIdx.x / LD, d = (threadIdx.x - grp * LD);
  griddep_wait();
  griddep_launch();
  const int n = paged_len(p, b);
  if (n == 0) {
    // no CTA of the split kernel meets an empty stream
    if (grp == 0) store_out4(p, row * D + 4 * d, make_float4(0.f, 0.f, 0.f, 0.f), 0.f);
    if (threadIdx.x == 0) {
      if (p.lse) p.lse[row] = -CUDART_INF_F;
      if (h == 0 && head == 0 && p.status && p.lens[b] != n) atomicOr(p.status, DEV_ERR_CHECK);
    }
    return;
  }
  const PagedShares shares(p, p.pre[p.B]);
  const int64_t load = paged_load(p, n);
  const int64_t first = p.pre[b] + h * load;
  const int i0 = shares.of(first + p.piece_load), i1 = shares.of(first + load - 1);
  if (i0 == i1) return;                        // written by its CTA
  float m = -CUDART_INF_F, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = i0 + grp; i <= i1; i += NG) {
    const int64_t part = (2 * (int64_t)i + (i == i0 ? 1 : 0)) * p.g + head;
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + part * 2);
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + part * D + 4 * d);
    const float mn = fmaxf(m, ml.x);
    const float f0 = m == mn ? 1.f : exp2f(m - mn), f1 = ml.x == mn ? 1.f : exp2f(ml.x - mn);
    l = l * f0 + ml.y * f1;
    o.x = o.x * f0 + v.x * f1;
    o.y = o.y * f0 + v.y * f1;
    o.z = o.z * f0 + v.z * f1;
    o.w = o.w * f0 + v.w * f1;
    m = mn;
  }
  so[grp][d] = o;
  if (d == 0) sm[grp] = m, sl[grp] = l;
  __syncthreads();
  if (grp == 0) {
    float top = sm[0];
#pragma unroll
    for (int k = 1; k < NG; ++k) top = fmaxf(top, sm[k]);
    float sum = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      const float f = sm[k] == top ? 1.f : exp2f(sm[k] - top);
      const float4 v = so[k][d];
      sum += sl[k] * f;
      a.x += v.x * f, a.y += v.y * f, a.z += v.z * f, a.w += v.w * f;
    }
    store_out4(p, row * D + 4 * d, a, sum == 0.f ? 0.f : 1.f / sum);
    if (d == 0) {
      store_stat(p, row, top, sum);
    }
  }
}

// ---------------------------------------------------------------------------
// weights: acc[t] += sum over the group of exp2(score - reference) / sum.  One owner per
// token: no atomics.  Memory-bound: 4 g bytes read and 8 read and written per
// token against 4 D for its fp16 rows (128K batch 8, group 4: 268 MB beside the
// 4.3 GB of keys and values).
// grid: streams * chunks of WT tokens
// ---------------------------------------------------------------------------
constexpr int WT = 1024;

__global__ void __launch_bounds__(JT) paged_weights_kernel(const __grid_constant__ PagedAttnParams p,
                                                           int chunks) {
  __shared__ float4 z[MAX_G];
  const int64_t stream = blockIdx.x / chunks;
  const int t = (int)(blockIdx.x - stream * chunks) * WT + threadIdx.x * 4;
  const int b = (int)(stream / p.H);
  griddep_wait();
  griddep_launch();
  const int n = paged_len(p, b);
  if (threadIdx.x < p.g) z[threadIdx.x] = p.stat[stream * p.g + threadIdx.x];
  __syncthreads();
  if (t >= n) return;
  float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* s = p.scores + stream * p.g * p.score_stride + t;
#pragma unroll 4
  for (int i = 0; i < p.g; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(s + i * p.score_stride);
    // a masked token weighs nothing, in a row without any live token too; the
    // difference to the reference comes first, so that no digit of a token that
    // weighs much is lost
    const float4 y = z[i];
    auto weight = [&](float x) { return x == -CUDART_INF_F ? 0.f : exp2f(fmaf(x, y.z, -y.x) - y.y); };
    w.x += weight(v.x);
    w.y += weight(v.y);
    w.z += weight(v.z);
    w.w += weight(v.w);
  }
  float* a = p.acc + stream * p.acc_stride + t;
  if (t + 4 <= n && (reinterpret_cast<uintptr_t>(a) & 15u) == 0) {
    float4 v = *reinterpret_cast<const float4*>(a);
    v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    *reinterpret_cast<float4*>(a) = v;
  } else {
    a[0] += w.x;
    if (t + 1 < n) a[1] += w.y;
    if (t + 2 < n) a[2] += w.z;
    if (t + 3 < n) a[3] += w.w;
  }
}

}  // namespace

namespace {

template <int D>
cudaError_t join_d(const PagedAttnParams& p, cudaStream_t st) {
  const int64_t rows = (int64_t)p.B * p.H * p.g;
  const dim3 grid((unsigned)rows);
  if (rows <= 2 * p.sms) return launch_kernel(paged_join_kernel<D, 1024>, grid, dim3(1024), 0, st, true, 0, p);
  return launch_kernel(paged_join_kernel<D, JT>, grid, dim3(JT), 0, st, true, 0, p);
}

}  // namespace

cudaError_t launch_paged_merge(const PagedAttnParams& p, int D, cudaStream_t st) {
  switch (D) {
    case 64: return join_d<64>(p, st);
    case 128: return join_d<128>(p, st);
    default: return join_d<256>(p, st);
  }
}

cudaError_t launch_paged_weights(const PagedAttnParams& p, cudaStream_t st) {
  const int chunks = (p.limit + WT - 1) / WT;
  return launch_kernel(paged_weights_kernel, dim3((unsigned)((int64_t)p.B * p.H * chunks)), dim3(JT), 0,
                       st, true, 0, p, chunks);
}

}  // namespace mkv
