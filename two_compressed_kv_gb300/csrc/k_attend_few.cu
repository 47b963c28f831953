// Attention of few queries, heads of 64 and 128.
#include "attend.cuh"

namespace mkv {

cudaError_t launch_attend_few(const AttendParams& p, cudaStream_t st) {
  return p.D == 64 ? launch_tiles<64, 1, true>(p, st) : launch_tiles<128, 1, true>(p, st);
}

}  // namespace mkv
