// The paged attention kernel with options: 8-bit pages, up to 8 columns.
#include "paged_attn.cuh"

namespace mkv {

cudaError_t launch_paged_opt(const PagedAttnParams& p, int D, cudaStream_t st) {
  switch (D) {
    case 64: return launch_pa<MKV_DT_E4M3, 64, false, true>(p, st);
    case 128: return launch_pa<MKV_DT_E4M3, 128, false, true>(p, st);
    default: return launch_pa<MKV_DT_E4M3, 256, false, true>(p, st);
  }
}

}  // namespace mkv
