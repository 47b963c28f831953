// Attention of few queries, heads of 256.
#include "attend.cuh"

namespace mkv {

cudaError_t launch_attend_few_256(const AttendParams& p, cudaStream_t st) { return launch_tiles<256, 1, true>(p, st); }

}  // namespace mkv
