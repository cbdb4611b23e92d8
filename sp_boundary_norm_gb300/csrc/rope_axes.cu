// Rotary positions: instances with a coordinate for each of several axes.
#include "rope.cuh"

namespace spb {

cudaError_t launch_rope_axes(const RopeAxesParams& p, int dtype, int vec, cudaStream_t st) {
  return launch_rope_of<true>(p, dtype, vec, st);
}

}  // namespace spb
