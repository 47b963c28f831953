// Internal declarations of the attention of many queries: prompts, and new tokens
// over the paged cache.
#pragma once

#include "paged_internal.cuh"

namespace mkv {

constexpr float AT_BIAS = 8.f;     // weights carry a factor 2^8 until the division by their sum
constexpr float AT_SLACK = 6.f;    // how far scores (log2) may pass the reference of the exponents: fp16 weights,
constexpr float AT_SLACK_BF16 = 24.f;   // bf16 ones, whose range is that of the sums (a bias by distance raises
                                        // the maximum in every block of a row's keys)

// Pairs of a sequence and a KV head whose CTAs are in one order: few, so that several CTAs
// share keys in L2; many, so that short prompts begin with all their long pieces.  Us of 8K
// prompts, batch 4, and of a ragged batch of 96 pairs with 8: 1542, 68; 16: 1550, 64; 32:
// 1605, 58; pair by pair: 1549, 68 (and one 2K prompt 54, 39 with any of these).
constexpr int AT_BUNDLE = 16;

// Keys of a block, the step of the pass over the keys: tensor memory holds two blocks'
// scores of every row tile and the outputs, and a thread a block of its row's scores, or
// with few rows a quarter (168 registers where a third warpgroup runs).
constexpr int attend_block(int D, int tiles, bool e4m3, bool few) {
  return D == 256 || tiles == 2 || (e4m3 && !few) ? 64 : 128;
}

// Keys whose weighted values tensor memory sums up by itself.  The products cut their sums off
// towards zero, which adds up: outputs of values of one sign come out too small by up to 6e-9 of
// themselves a key (131072 keys: 8e-4, more than half a step of fp16).  So after AT_FOLD keys the
// sums are added to those in the workspace, with rounding to nearest, and begin again: 1e-4.  (8192
// keys: 5e-5, but 512 queries over 32768 keys take 203 us instead of 197.)
// Kernels of capped or biased scores have no registers for that (4096 x 2 tokens, capped: 312 us,
// 291 without; a ragged batch with a bias 58, 53): their keys are cut into parts of at most
// AT_PART, up to 64 of them, which the join adds: 2e-4.
constexpr int AT_FOLD = 16384, AT_PART = 32768;

struct AttendParams {
  const void* q;
  void* out;
  float* lse;                  // [B][nq][Hq], or NULL
  int64_t qs[3], os[3];        // elements between batches, tokens, heads
  int B, Hq, H, g, D;
  int nq;                      // queries of the longest sequence
  int nk;                      // bound on keys
  int bf16;                    // queries' type, else fp16
  const int32_t *q_lens, *kv_lens;   // or NULL: nq, nk
  const int32_t* prefix;
  const int32_t* docs;
  int64_t docs_stride;
  int2* doc_range;             // workspace: [B][blocks of keys] smallest and largest document
  const uint64_t* tree;
  const float* slopes;
  int causal, window;
  float scale, cap;
  int32_t* status;
  // keys in tensors
  const void *k, *v;
  int64_t ks[3], vs[3];
  // or in pages
  const int32_t* table;        // NULL: tensors
  int64_t table_stride;
  int n_pages, page_size, cache_type;
  const float *k_scale, *v_scale;
  // the grid: row tiles of a (sequence, KV head) in groups of `tiles`, their keys in `splits` parts
  int copies;                  // of its rows that a row tile holds: 1, or with few rows 2 or 4
  int tile_tokens;             // tokens of a row tile: 128 / copies / g
  int tiles;                   // row tiles of a CTA: 1 or 2
  int groups;                  // of row tiles
  int splits;
  int fold;                    // AT_FOLD in blocks, less 1; INT32_MAX where no walk is as long
  float4* part_o;              // workspace: [CTA][tiles][D / 4][128 rows] sums over weights, splits > 1 or fold
  float2* part_ml;             // [CTA][tiles][128] reference (log2 domain) and sum of weights
};

// What a sequence's lengths come to: queries and keys, both within their bounds.
__device__ __forceinline__ void attend_lens(const AttendParams& p, int b, int& m, int& L, bool& outside) {
  const int k = p.kv_lens ? p.kv_lens[b] : p.nk, q = p.q_lens ? p.q_lens[b] : p.nq;
  L = max(0, min(k, p.nk));
  m = max(0, min(q, p.nq));
  if (p.table) m = min(m, L);
  outside = L != k || (p.q_lens && m != q);
}

cudaError_t launch_attend_64(const AttendParams& p, cudaStream_t st);
cudaError_t launch_attend_128(const AttendParams& p, cudaStream_t st);
cudaError_t launch_attend_256(const AttendParams& p, cudaStream_t st);
cudaError_t launch_attend_2(const AttendParams& p, cudaStream_t st);        // two copies, 8-bit pages
cudaError_t launch_attend_4(const AttendParams& p, cudaStream_t st);        // four copies, heads of 64 and 128
cudaError_t launch_attend_4_256(const AttendParams& p, cudaStream_t st);
cudaError_t launch_attend_docs(const AttendParams& p, cudaStream_t st);
cudaError_t launch_attend_join(const AttendParams& p, cudaStream_t st);

// A tensor map of up to four dimensions (the first contiguous, strides in bytes), 128-byte swizzled or not.
cudaError_t encode_map(CUtensorMap* map, const void* base, bool bytes, int rank, const uint64_t* dim,
                       const uint64_t* stride, const uint32_t* box, bool swizzle);

}  // namespace mkv
