// Internal declarations of the attention of many queries: prompts, and new tokens
// over the paged cache.
#pragma once

#include "paged_internal.cuh"

namespace mkv {

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
  const uint64_t* tree;
  const float* slopes;
  int causal, window;
  float scale, cap;
  // keys in tensors
  const void *k, *v;
  int64_t ks[3], vs[3];
  // or in pages
  const int32_t* table;        // NULL: tensors
  int64_t table_stride;
  int n_pages, page_size, cache_type;
  const float *k_scale, *v_scale;
  int32_t* status;
};

cudaError_t launch_attend(const AttendParams& p, cudaStream_t st);

}  // namespace mkv
