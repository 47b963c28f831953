// Attention of few queries, 4 copies of their rows, heads of 256.
#include "attend.cuh"

namespace mkv {

cudaError_t launch_attend_4_256(const AttendParams& p, cudaStream_t st) { return launch_from<256, 1, 4>(p, st); }

}  // namespace mkv
