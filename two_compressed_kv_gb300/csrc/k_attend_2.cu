// Attention of few queries over 8-bit pages, two copies of their rows.
#include "attend.cuh"

namespace mkv {

cudaError_t launch_attend_2(const AttendParams& p, cudaStream_t st) {
  switch (p.D) {
    case 64: return launch_options<64, 1, FROM_BYTES, 2>(p, st);
    case 128: return launch_options<128, 1, FROM_BYTES, 2>(p, st);
    default: return launch_options<256, 1, FROM_BYTES, 2>(p, st);
  }
}

}  // namespace mkv
