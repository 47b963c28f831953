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

// A row's parts, in their order: weights' sums and outputs over a common reference.  A
// thread takes 16 channels of a row, a block the rows of a tile, so that the parts are
// read a line at a time.  grid: (row tiles, D / 16)
template <int D>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ AttendParams p) {
  griddep_wait();
  griddep_launch();
  const int row = threadIdx.x, per = p.groups * p.tiles;
  const int64_t bh = div_small(blockIdx.x, per);
  const int all = (int)(blockIdx.x - bh * per), b = (int)(bh / p.H), h = (int)(bh - (int64_t)b * p.H);
  const int rt = row / p.g, token = all * p.tile_tokens + rt, head = h * p.g + row - rt * p.g;
  int m, L;
  bool outside;
  attend_lens(p, b, m, L, outside);
  if (rt >= p.tile_tokens || token >= m) return;
  const int group = all / p.tiles, tile = all - group * p.tiles;
  // CTA of part 0; the groups run backwards
  const int64_t first = ((bh * p.groups + p.groups - 1 - group) * p.splits) * p.tiles + tile;
  const float2* ml = p.part_ml + first * 128 + row;
  const float4* part = p.part_o + (first * (D / 4) + blockIdx.y * 4) * 128 + row;
  const int64_t ml_step = (int64_t)p.tiles * 128, step = ml_step * (D / 4);
  float top = -CUDART_INF_F;
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, ml[s * ml_step].x);
  float sum = 0.f;
  float4 o[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int s = 0; s < p.splits; ++s) {
    const float2 x = ml[s * ml_step];
    const float f = x.x == top ? 1.f : x.x == -CUDART_INF_F ? 0.f : exp2f(x.x - top);
    sum += x.y * f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 v = part[s * step + c * 128];
      o[c].x += v.x * f, o[c].y += v.y * f, o[c].z += v.z * f, o[c].w += v.w * f;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* out = static_cast<uint16_t*>(p.out) + b * p.os[0] + (int64_t)token * p.os[1] + head * p.os[2] + blockIdx.y * 16;
  uint32_t u[8];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float4 v = make_float4(o[c].x * inv, o[c].y * inv, o[c].z * inv, o[c].w * inv);
    if (p.bf16) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
      u[2 * c] = *reinterpret_cast<const uint32_t*>(&x), u[2 * c + 1] = *reinterpret_cast<const uint32_t*>(&y);
    } else {
      const __half2 x = __floats2half2_rn(v.x, v.y), y = __floats2half2_rn(v.z, v.w);
      u[2 * c] = *reinterpret_cast<const uint32_t*>(&x), u[2 * c + 1] = *reinterpret_cast<const uint32_t*>(&y);
    }
  }
  reinterpret_cast<uint4*>(out)[0] = make_uint4(u[0], u[1], u[2], u[3]);
  reinterpret_cast<uint4*>(out)[1] = make_uint4(u[4], u[5], u[6], u[7]);
  if (p.lse && blockIdx.y == 0)
    p.lse[((int64_t)b * p.nq + token) * p.Hq + head] =
        sum == 0.f ? -CUDART_INF_F : (top + (log2f(sum) - AT_BIAS)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_attend_docs(const AttendParams& p, cudaStream_t st) {
  const int block = attend_block(p.D, p.tiles, false, p.copies > 1), blocks = (p.nk + block - 1) / block;
  if (blocks == 0) return cudaSuccess;
  return launch_kernel(docs_kernel, dim3((blocks + 3) / 4, p.B), dim3(128), 0, st, true, 0, p, block, blocks);
}

cudaError_t launch_attend_join(const AttendParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)((int64_t)p.B * p.H * p.groups * p.tiles), p.D / 16), block(128);
  switch (p.D) {
    case 64: return launch_kernel(join_kernel<64>, grid, block, 0, st, true, 0, p);
    case 128: return launch_kernel(join_kernel<128>, grid, block, 0, st, true, 0, p);
    default: return launch_kernel(join_kernel<256>, grid, block, 0, st, true, 0, p);
  }
}

}  // namespace mkv
