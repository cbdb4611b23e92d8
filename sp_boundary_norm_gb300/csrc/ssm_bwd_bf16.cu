// Selective scan, backward: instances of one element type.
#include "ssm_bwd.cuh"

namespace spb {

template cudaError_t launch_ssm_bwd_of<SP_BF16>(const SsmParams&, const SsmParamGrads&, cudaStream_t);

}  // namespace spb
