// Attention of few queries, 4 copies of their rows, heads of 64 and 128.
#include "attend.cuh"

namespace mkv {

cudaError_t launch_attend_4(const AttendParams& p, cudaStream_t st) {
  return p.D == 64 ? launch_from<64, 1, 4>(p, st) : launch_from<128, 1, 4>(p, st);
}

}  // namespace mkv
