// The paged attention kernel at head dimension 64.
#include "paged_attn.cuh"

namespace mkv {

cudaError_t launch_paged_attn_64(const PagedAttnParams& p, int cache_type, cudaStream_t st) {
  return launch_pa_d<64>(p, cache_type, st);
}

}  // namespace mkv
