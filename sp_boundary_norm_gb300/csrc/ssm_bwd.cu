// Selective scan, backward: launches.
#include "ssm_bwd.cuh"

namespace spb {

template <int DT, int N>
static cudaError_t launch_bwd(const SsmParams& p, const SsmParamGrads& g, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (p.chunks > 1) {
    e = launch_walk<DT, N, kSsmBack>(p, st);
    if (e == cudaSuccess) e = launch_join<true>(p, st);
    if (e != cudaSuccess) return e;
  }
  e = launch_back<DT, N>(p, st);
  if (e == cudaSuccess && p.partial_bc != nullptr) {
    void* args[] = {const_cast<SsmParams*>(&p)};
    const int64_t threads = static_cast<int64_t>(p.b) * p.s * (p.n / 2) * p.t * p.groups;
    e = launch_pdl(reinterpret_cast<const void*>(&ssm_bc_kernel<DT>),
                   dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, args, st);
  }
  if (e == cudaSuccess && p.partial_params != nullptr) {
    const float* from = p.partial_params;
    int64_t channels = static_cast<int64_t>(p.t) * p.c, parts = static_cast<int64_t>(p.b) * p.chunks;
    int n = p.n;
    SsmParamGrads grads = g;
    void* args[] = {&from, &channels, &n, &parts, &grads};
    const int64_t columns = channels * (n + 2);
    e = launch_pdl(reinterpret_cast<const void*>(&ssm_params_kernel),
                   dim3(static_cast<unsigned>((columns + 31) / 32)), dim3(kPartThreads), 0, args, st);
  }
  return e;
}

template <int DT>
static cudaError_t launch_states(const SsmParams& p, const SsmParamGrads& g, cudaStream_t st) {
  switch (p.n) {
    case 8: return launch_bwd<DT, 8>(p, g, st);
    case 16: return launch_bwd<DT, 16>(p, g, st);
    case 32: return launch_bwd<DT, 32>(p, g, st);
    default: return launch_bwd<DT, 64>(p, g, st);
  }
}

cudaError_t launch_ssm_bwd(const SsmParams& p, int dtype, const SsmParamGrads& g,
                           cudaStream_t st) {
  return dtype == SP_BF16  ? launch_states<SP_BF16>(p, g, st)
         : dtype == SP_F16 ? launch_states<SP_F16>(p, g, st)
                           : launch_states<SP_F32>(p, g, st);
}

}  // namespace spb
