// Attention of many queries, heads of 64.
#include "attend.cuh"

namespace mkv {

cudaError_t launch_attend_64(const AttendParams& p, cudaStream_t st) {
  return launch_attend_d<64>(p, st);
}

}  // namespace mkv
