// What the host sides of the rotary, paged-cache and prompt calls share.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstring>

#include "paged_internal.cuh"

namespace mkv {

constexpr int64_t kMaxGrid = 0x7fffffff;

#define CKP(call)                                              \
  do {                                                         \
    cudaError_t e_ = (call);                                   \
    if (e_ != cudaSuccess) return set_cuda_error(e_, #call);   \
  } while (0)

inline mkv_status bad(const char* text) { return set_error(MKV_ERR_INVALID_ARG, text); }

inline int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool is16(int dtype) { return dtype == MKV_DT_F16 || dtype == MKV_DT_BF16; }
// Stride of a dimension that is walked over: 16-byte accesses need multiples of 8
// elements.  That of an extent of 1 is never used.
inline bool stride8(int64_t stride, int64_t extent) { return extent <= 1 || stride % 8 == 0; }
inline int elem_bytes(int dtype) { return dtype == MKV_DT_F32 ? 4 : dtype == MKV_DT_E4M3 ? 1 : 2; }

// SMs of the current device.
mkv_status sm_count(int* out);

// Heads a thread takes so that its angles serve several heads while the grid
// still has at least `want` threads.
int heads_per_thread(int64_t threads, int heads, int64_t want, int most);

// What is wrong with a plan, its axes or a cache view; NULL: nothing.
const char* check_plan(const mkv_rope_plan* p);
const char* check_axes(const mkv_rope_axes* x, const mkv_rope_plan* p);
const char* check_cache(const mkv_paged_cache* c);

// Few new tokens over 8-bit pages, by the streaming kernel of the single token: whether a
// call is such a one.  Arguments have been checked; workspace: bytes, and whether the
// caller's is enough.
bool paged_attend_streams(const mkv_paged_cache* c, const mkv_paged_attend_args* a);
mkv_status paged_attend_streaming(const mkv_paged_cache* c, const mkv_paged_attend_args* a, mkv_stream_t stream);
uint64_t paged_attend_streaming_workspace(const mkv_paged_cache* c, const mkv_paged_attend_args* a);

}  // namespace mkv
