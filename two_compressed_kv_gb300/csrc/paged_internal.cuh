// Internal declarations of the rotary and paged-cache operators.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mkv.h"
#include "mkv_internal.cuh"

namespace mkv {

// Sets the text that mkv_last_error_string returns; `s` is passed through.
mkv_status set_error(mkv_status s, const char* text) noexcept;
mkv_status set_cuda_error(cudaError_t e, const char* what) noexcept;

// ---------------------------------------------------------------------------
// rope and append
// ---------------------------------------------------------------------------
struct RopeParams {
  mkv_rope_plan plan;
  const void* x;
  void* out;
  const int32_t* pos;
  int64_t xs[3], os[3], pos_stride;
  int64_t tokens;
  int batch, heads;
  int first_pos;
  int units;          // per head: work of one thread (a vector pair, a vector, a pair or an element)
  int rot_units;      // those that rotate; the rest copy
  int heads_per;      // heads a thread handles
  float sign;         // -1: transposed
};
cudaError_t launch_rope(const RopeParams& p, int dtype, bool vec, cudaStream_t st);

struct AppendRowsParams {
  mkv_rope_plan plan;             // rot_dim 0: no rotation
  mkv_paged_cache c;
  mkv_paged_append_args a;
  int units, rot_units, heads_per, heads_total;
};
cudaError_t launch_append_rows(const AppendRowsParams& p, cudaStream_t st);

// ---------------------------------------------------------------------------
// attention over the paged cache
// ---------------------------------------------------------------------------
constexpr int PA_BLOCK = 16;      // tokens per block: the unit of work; a block lies in one page
constexpr int PA_MAX_B = 512;     // sequences whose prefix sums fit the split kernel
constexpr float PA_SLACK = 3.f;    // how far scores (log2) may pass the reference of the exponents
constexpr float PA_UNSET = 1e38f;
constexpr float PA_BIAS = 12.f;   // probabilities carry a factor 2^12 until the division by their sum

// CTAs of the streaming kernel per SM, by the bytes of a row: its rings and
// accumulators grow with the row, and with short rows the latency of a step
// counts more.
constexpr int paged_ctas(int row_bytes) { return row_bytes >= 512 ? 1 : row_bytes >= 256 ? 2 : 3; }

struct PagedAttnParams {
  const uint8_t *kp, *vp;
  const int32_t* table;
  const float *ks, *vs;
  int32_t* status;
  int64_t table_stride;
  int64_t rows;                   // of a pool: n_pages * H * page_size
  int B, H, g, n_pages, bpp;      // bpp: blocks per page
  int limit;                      // largest length: min(max_len, max_pages * page_size)
  const void* q;
  int64_t q_sb, q_sh;
  int q_bf16;
  void* out;
  int out_type;                   // MKV_DT_*
  float* lse;
  const int32_t* lens;
  float scale2;                   // scale * log2(e)
  float* acc;
  int64_t acc_stride;
  // workspace
  float* part_o;                  // [6 G][g][D]: unnormalised sums of split streams
  float* part_ml;                 // [6 G][g][2]: running maximum (log2 domain) and sum
  float4* stat;                   // [B H g]: reference of the exponents and log2 of the sum over it, in
                                  // the scaled log2 domain; scale of the kept scores
  int64_t* pre;                   // [B + 1]: load before each sequence (split)
  float* scores;                  // [B H g][score_stride], unscaled; only with acc
  int64_t score_stride;
  int sms;                        // of the device
  int G;                          // large shares of the split kernel; 2 G small ones follow
  int min_blocks;                 // smallest share of a CTA, in blocks
  int piece_load;                 // what a part of a stream costs apart from its blocks, in blocks
  int tail16;                     // sixteenths of the load that are handed out in small shares
  int tail_from;                  // from this many blocks a CTA on
  int split;                      // 0: a cluster of CTAs per stream
  int cluster;                    // its size, 1 to 8 (split: 1)
};

// Cached tokens of sequence b as the kernels count them.
__device__ __forceinline__ int paged_len(const PagedAttnParams& p, int b) {
  const int n = p.lens[b];
  return n < 0 ? 0 : min(n, p.limit);
}

// a / b, mostly of numbers that fit 32 bits (a 64-bit division is some hundred
// instructions in a prologue that every share pays).
__device__ __forceinline__ int64_t div_small(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Load of a stream of n tokens: its blocks and a fixed cost.
__device__ __forceinline__ int64_t paged_load(const PagedAttnParams& p, int n) {
  return n == 0 ? 0 : (n + PA_BLOCK - 1) / PA_BLOCK + p.piece_load;
}

// How the split kernel's CTAs share the load of all streams: the first G, which
// run at once, take equal large shares, and 2 G more take what is left in
// small ones as SMs become free, so that an SM that gets less of the memory's
// bandwidth than others does not finish late.  A function of the lengths alone.
constexpr int PA_SHARES = 3;
struct PagedShares {
  int64_t total, big, small;
  int G;
  __device__ __forceinline__ PagedShares(const PagedAttnParams& p, int64_t total_) : total(total_), G(p.G) {
    if (total < (int64_t)G * p.tail_from) {
      big = max(div_small(total + G - 1, G), (int64_t)p.min_blocks);
      small = 1;
    } else {
      big = div_small(total * (16 - p.tail16) / 16, G);
      small = div_small(total - big * G + 2 * G - 1, 2 * G);
    }
  }
  // start of share i, and the share that load v belongs to
  __device__ __forceinline__ int64_t first(int64_t i) const {
    return min(total, i < G ? i * big : G * big + (i - G) * small);
  }
  __device__ __forceinline__ int of(int64_t v) const {
    return (int)(v < G * big ? div_small(v, big) : G + div_small(v - G * big, small));
  }
};

// Four outputs a * f from element `at` on, rounded to the output's type.
__device__ __forceinline__ void store_out4(const PagedAttnParams& p, int64_t at, float4 a, float f) {
  a.x *= f, a.y *= f, a.z *= f, a.w *= f;
  if (p.out_type == MKV_DT_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = a;
  } else if (p.out_type == MKV_DT_BF16) {
    __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + at);
    o[0] = __floats2bfloat162_rn(a.x, a.y);
    o[1] = __floats2bfloat162_rn(a.z, a.w);
  } else {
    __half2* o = reinterpret_cast<__half2*>(static_cast<__half*>(p.out) + at);
    o[0] = __floats2half2_rn(a.x, a.y);
    o[1] = __floats2half2_rn(a.z, a.w);
  }
}

// Tensor map of a pool as [rows][row_bytes]: copies of `box_rows` whole rows,
// laid out [row_bytes / w][box_rows][w] with w = min(row_bytes, 128), swizzled
// over w bytes.
cudaError_t encode_rows_map(CUtensorMap* map, const void* base, int64_t rows, int row_bytes, int box_rows);

// Statistics of a finished row (d == 0's thread): the sum of exp2(score - top + PA_BIAS).
__device__ __forceinline__ void store_stat(const PagedAttnParams& p, int64_t row, float top, float sum) {
  const float lg = log2f(sum) - PA_BIAS;
  if (p.lse) p.lse[row] = sum == 0.f ? __int_as_float(0xff800000) : (top + lg) * 0.6931471805599453f;
  if (p.scores) *reinterpret_cast<float2*>(p.stat + row) = make_float2(top, lg);
}

// g <= 8 and g <= 16 variants per head dim (one translation unit each)
cudaError_t launch_paged_attn_64(const PagedAttnParams& p, int cache_type, cudaStream_t st);
cudaError_t launch_paged_attn_128(const PagedAttnParams& p, int cache_type, cudaStream_t st);
cudaError_t launch_paged_attn_256(const PagedAttnParams& p, int cache_type, cudaStream_t st);
cudaError_t launch_paged_merge(const PagedAttnParams& p, int D, cudaStream_t st);
cudaError_t launch_paged_weights(const PagedAttnParams& p, cudaStream_t st);

// ---------------------------------------------------------------------------
// eviction
// ---------------------------------------------------------------------------
struct EvictParams {
  uint8_t *kp, *vp;
  const int32_t* table;
  int32_t* status;
  int64_t table_stride;
  int B, H, n_pages, ps, row_bytes;
  int limit;
  const float* acc;
  const int32_t* pos;
  float* acc_out;
  int32_t* pos_out;
  const int32_t *lens, *next_pos;
  int32_t *lens_out, *src;
  int64_t meta_stride, out_stride;
  int budget, sink, recent;
  int32_t* lists;                 // workspace: [B H][2][budget] movers, then holes (budget < limit)
  uint2* listed;                  // workspace: [B H][list_slots] (key, slot), long slices only
  int64_t list_slots;
  int R;                          // CTAs (one cluster) per stream
};
// Entries of `listed` a stream needs: 0 where slices are short.
int64_t evict_list_slots(int64_t limit, int R);
cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t st);
cudaError_t launch_evict_move(const EvictParams& p, cudaStream_t st);

}  // namespace mkv
