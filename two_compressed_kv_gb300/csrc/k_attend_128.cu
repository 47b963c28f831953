// Attention of many queries, heads of 128.
#include "attend.cuh"

namespace mkv {

cudaError_t launch_attend_128(const AttendParams& p, cudaStream_t st) {
  return launch_attend_d<128>(p, st);
}

}  // namespace mkv
