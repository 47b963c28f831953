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

// With several axes: pos is [axes][batch][tokens].
struct RopeMultiParams : RopeParams {
  mkv_rope_axes axes;
  int64_t pos_axis_stride;
};
cudaError_t launch_rope_multi(const RopeMultiParams& p, int dtype, bool vec, cudaStream_t st);

// Norms of heads and their rotation.
struct NormRopeParams {
  mkv_rope_plan plan;
  mkv_rope_axes axes;               // n_axes 0: one position a token, from pos or first_pos
  const void *x[2], *grad[2], *weight[2];
  void* out[2];
  int64_t xs[2][3], os[2][3], gs[2][3];
  const int32_t* pos;
  int64_t pos_stride, pos_axis_stride;
  int64_t tokens, items[2];         // a side's items: batch * tokens * chunks
  int batch, heads[2], first_pos;
  int weight_f32[2];                // the weight's type (0: x's)
  float eps, offset;
  int units, rot_units;             // of a head, as in RopeParams
  int lanes;                        // that share a head: a power of two up to 32
  int heads_per, chunks[2];         // heads a group of lanes takes
  int blocks[2];                    // of each side
  float* part;                      // gradient: [blocks][head_dim] sums of a block, or NULL
  float* weight_grad[2];
};
// Bytes of the vectors that a lane takes of a head.  The gradient holds four times as many
// values as the norm, so of 16-bit heads it takes half: 84 us with 8 bytes, 97 with 16.
constexpr int norm_vector_bytes(bool is16, bool grad) { return is16 && grad ? 8 : 16; }
// form: 0 elements, 1 vectors of half pairs, 2 vectors of interleaved pairs
cudaError_t launch_norm_rope(const NormRopeParams& p, int dtype, int form, bool grad, cudaStream_t st);

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
  // Several new tokens, scores with options (kernels with OPT): the g "heads" of a stream are
  // its new tokens times their heads.
  int opt;
  int tokens, heads;              // g = tokens * heads
  int64_t q_st;                   // elements between tokens of q
  const int32_t* new_lens;        // or NULL: tokens
  const uint64_t* tree;           // or NULL: a chain
  const float* slopes;
  int window;
  float cap2;                     // cap * log2(e); 0: none
};

// Cached and new tokens of sequence b with options, both within their bounds, and the
// first block that one of the new tokens sees.
struct PagedReach {
  int n, m, first;
  bool outside;
  __device__ __forceinline__ PagedReach(const PagedAttnParams& p, int b) {
    const int k = p.lens[b], q = p.new_lens ? p.new_lens[b] : p.tokens;
    n = max(0, min(k, p.limit));
    m = max(0, min(min(q, p.tokens), n));
    outside = k != n || (p.new_lens && q != m);
    first = p.window ? max(0, n - m - p.window + 1) / PA_BLOCK : 0;
    if (m == 0) n = first = 0;    // nothing to attend for
  }
};
// Row of the output for column `col` of stream (b, h).
__device__ __forceinline__ int64_t paged_row(const PagedAttnParams& p, int64_t b, int h, int col) {
  const int t = col / p.heads;
  return (b * p.tokens + t) * (p.H * p.heads) + h * p.heads + col - t * p.heads;
}

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
__device__ __forceinline__ int64_t paged_load(const PagedAttnParams& p, int n, int first = 0) {
  return n == 0 ? 0 : (n + PA_BLOCK - 1) / PA_BLOCK - first + p.piece_load;
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

// cap tanh(z / cap) of a score in the log2 domain, cap2 its cap there.  Up to half the cap z
// times a polynomial in (z / cap)^2 with the smallest largest relative error (found by
// exchange): the error goes by z and not by the cap, however large that is.  Beyond it
// 1 - 2 / (e + 1), whose error is one of the cap's last bits.  Within 2^-20 of the result.
struct CappedScore {
  float cap2, over;                // over: 1 / cap2, finite
  __device__ __forceinline__ explicit CappedScore(float cap2_) : cap2(cap2_), over(fminf(1.f / cap2_, 3.402823466e38f)) {}
  // |z| <= cap2 / 2
  __device__ __forceinline__ float small(float z) const {
    const float t = z * over, u = t * t;
    float y = fmaf(u, 0.017135007306933403f, -0.05298607423901558f);
    y = fmaf(u, y, 0.13324779272079468f);
    y = fmaf(u, y, -0.3333306908607483f);
    return z * fmaf(u, y, 1.f);
  }
  // x: 2 log2(e) times z / cap
  __device__ __forceinline__ float large(float x) const {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e) : "f"(fabsf(x)));
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(e + 1.f));
    return cap2 * copysignf(fmaf(-2.f, r, 1.f), x);
  }
  __device__ __forceinline__ float operator()(float z) const {
    return fabsf(z) <= 0.5f * cap2 ? small(z) : large(z * over * 2.885390081777927f);
  }
};

// g <= 8 and g <= 16 variants per head dim (one translation unit each)
cudaError_t launch_paged_attn_64(const PagedAttnParams& p, int cache_type, cudaStream_t st);
cudaError_t launch_paged_attn_128(const PagedAttnParams& p, int cache_type, cudaStream_t st);
cudaError_t launch_paged_attn_256(const PagedAttnParams& p, int cache_type, cudaStream_t st);
cudaError_t launch_paged_opt(const PagedAttnParams& p, int D, cudaStream_t st);   // E4M3, g <= 8
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
