// Attention of many queries, heads of 256.
#include "attend.cuh"

namespace mkv {

cudaError_t launch_attend_256(const AttendParams& p, cudaStream_t st) {
  return launch_attend_d<256>(p, st);
}

}  // namespace mkv
