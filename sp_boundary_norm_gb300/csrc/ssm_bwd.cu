// Selective scan, backward: the element type's launches.
#include "region.h"

namespace spb {

template <int DT>
cudaError_t launch_ssm_bwd_of(const SsmParams& p, const SsmParamGrads& g, cudaStream_t st);

cudaError_t launch_ssm_bwd(const SsmParams& p, int dtype, const SsmParamGrads& g,
                           cudaStream_t st) {
  return dtype == SP_BF16  ? launch_ssm_bwd_of<SP_BF16>(p, g, st)
         : dtype == SP_F16 ? launch_ssm_bwd_of<SP_F16>(p, g, st)
                           : launch_ssm_bwd_of<SP_F32>(p, g, st);
}

}  // namespace spb
