// Rotary positions: instances with one position a token.
#include "rope.cuh"

namespace spb {

cudaError_t launch_rope(const RopeParams& p, int dtype, int vec, cudaStream_t st) {
  return launch_rope_of<false>(p, dtype, vec, st);
}

}  // namespace spb
