// The paged attention kernel at head dimension 128.
#include "paged_attn.cuh"

namespace mkv {

cudaError_t launch_paged_attn_128(const PagedAttnParams& p, int cache_type, cudaStream_t st) {
  return launch_pa_d<128>(p, cache_type, st);
}

}  // namespace mkv
