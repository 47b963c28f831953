// Around the attention of many queries: the documents' range in every block of keys
// before it, and the join of the parts of a row's keys after it.
#include <math_constants.h>

#include "attend_internal.cuh"
#include "decode_common.cuh"

namespace mkv {
namespace {

// grid: (blocks of keys / 4, B); a warp a block
__global__ void __launch_bounds__(128) docs_kernel(const __grid_constant__ AttendParams p, int block, int blocks) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, j = blockIdx.x * 4 + (threadIdx.x >> 5), b = blockIdx.y;
  if (j >= blocks) return;
  const int32_t* docs = p.docs + b * p.docs_stride;
  int least = INT32_MAX, most = INT32_MIN;
  for (int t = j * block + lane; t < min(p.nk, (j + 1) * block); t += 32) {
    least = min(least, docs[t]);
    most = max(most, docs[t]);
  }
  least = __reduce_min_sync(~0u, least);
  most = __reduce_max_sync(~0u, most);
  if (lane == 0) p.doc_range[(int64_t)b * blocks + j] = make_int2(least, most);
}

// A row's parts, in their order: weights' sums and outputs over a common reference.
// A warp a row; grid: B * nq * Hq / 4.
template <int D>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ AttendParams p) {
  griddep_wait();
  griddep_launch();
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (id >= (int64_t)p.B * p.nq * p.Hq) return;
  const int64_t bt = div_small(id, p.Hq);
  const int head = (int)(id - bt * p.Hq), b = (int)div_small(bt, p.nq), token = (int)(bt - (int64_t)b * p.nq);
  int m, L;
  bool outside;
  attend_lens(p, b, m, L, outside);
  if (token >= m) return;
  const int h = head / p.g, all = token / p.tile_tokens, row = (token - all * p.tile_tokens) * p.g + head - h * p.g;
  const int group = all / p.tiles, tile = all - group * p.tiles;
  // CTA of part 0; the groups run backwards
  const int64_t cta = (((int64_t)b * p.H + h) * p.groups + p.groups - 1 - group) * p.splits;
  const int64_t first = (cta * p.tiles + tile) * 128 + row, step = (int64_t)p.tiles * 128;
  float top = -CUDART_INF_F;
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, p.part_ml[first + s * step].x);
  float sum = 0.f, o[N];
#pragma unroll
  for (int c = 0; c < N; ++c) o[c] = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float2 ml = p.part_ml[first + s * step];
    const float f = ml.x == top ? 1.f : ml.x == -CUDART_INF_F ? 0.f : exp2f(ml.x - top);
    const float* from = p.part_o + (first + s * step) * D + lane * N;
    sum += ml.y * f;
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const float2 v = *reinterpret_cast<const float2*>(from + c);
      o[c] += v.x * f;
      o[c + 1] += v.y * f;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* out = static_cast<uint16_t*>(p.out) + b * p.os[0] + (int64_t)token * p.os[1] + head * p.os[2] + lane * N;
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    if (p.bf16) *reinterpret_cast<__nv_bfloat162*>(out + c) = __floats2bfloat162_rn(o[c] * inv, o[c + 1] * inv);
    else *reinterpret_cast<__half2*>(out + c) = __floats2half2_rn(o[c] * inv, o[c + 1] * inv);
  }
  if (p.lse && lane == 0)
    p.lse[id] = sum == 0.f ? -CUDART_INF_F : (top + (log2f(sum) - AT_BIAS)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_attend_docs(const AttendParams& p, cudaStream_t st) {
  const int block = attend_block(p.D, p.tiles, false, p.few), blocks = (p.nk + block - 1) / block;
  if (blocks == 0) return cudaSuccess;
  return launch_kernel(docs_kernel, dim3((blocks + 3) / 4, p.B), dim3(128), 0, st, true, 0, p, block, blocks);
}

cudaError_t launch_attend_join(const AttendParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)(((int64_t)p.B * p.nq * p.Hq + 3) / 4)), block(128);
  switch (p.D) {
    case 64: return launch_kernel(join_kernel<64>, grid, block, 0, st, true, 0, p);
    case 128: return launch_kernel(join_kernel<128>, grid, block, 0, st, true, 0, p);
    default: return launch_kernel(join_kernel<256>, grid, block, 0, st, true, 0, p);
  }
}

}  // namespace mkv
