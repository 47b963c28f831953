// The paged attention kernel at head dimension 256.
#include "paged_attn.cuh"

namespace mkv {

cudaError_t launch_paged_attn_256(const PagedAttnParams& p, int cache_type, cudaStream_t st) {
  return launch_pa_d<256>(p, cache_type, st);
}

}  // namespace mkv
