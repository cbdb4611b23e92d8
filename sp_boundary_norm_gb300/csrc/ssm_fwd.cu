// Selective scan, forward: launches of the walk.
#include "ssm_fwd.cuh"

namespace spb {

template <int DT, int N>
static cudaError_t launch_fwd(const SsmParams& p, cudaStream_t st) {
  if (p.chunks > 1) {
    cudaError_t e = launch_walk<DT, N, kSsmEnds>(p, st);
    if (e == cudaSuccess) e = launch_join<false>(p, st);
    if (e != cudaSuccess) return e;
  }
  return launch_walk<DT, N, kSsmOut>(p, st);
}

template <int DT>
static cudaError_t launch_states(const SsmParams& p, cudaStream_t st) {
  switch (p.n) {
    case 8: return launch_fwd<DT, 8>(p, st);
    case 16: return launch_fwd<DT, 16>(p, st);
    case 32: return launch_fwd<DT, 32>(p, st);
    default: return launch_fwd<DT, 64>(p, st);
  }
}

constexpr int64_t kMostChunks = 160;

SsmSplit ssm_split(int64_t b, int64_t s, int64_t c, int n, int groups, int t, bool bwd) {
  const int block = n <= 16 ? 64 : n == 32 ? 32 : 16;
  const int64_t of_group = c / groups;
  SsmSplit k{};
  k.slabs = static_cast<int32_t>((of_group + block - 1) / block);
  const int64_t blocks = b * t * groups * k.slabs, sms = device_sm_count();
  // A block has an SM to itself, so a call takes as many waves of blocks as they need, each
  // as long as a chunk and some 48 tokens' time to begin.  Chunks cost a walk for what
  // enters them, 75 clocks a token beside the forward's 132 and the backward's 447, two
  // launches, and their joining.  (Measured: 8 x 8192 x 1024, 128 blocks, forward 531 us
  // whole, 675 cut; 32,769 x 512, 8 blocks that would walk 2.0 ms, cut
  // in 19 191 us; 256 x 64, forward and backward in two chunks 18 and 38 us, in 16 10 and 17.)
  const double walk = bwd ? 1.2 : 1.6, start = bwd ? 15 : 50, join = bwd ? 6 : 16;
  double least = 0;
  for (int64_t n = 1; n <= kMostChunks && (n == 1 || n * kSsmTile <= s); ++n) {
    const int64_t len = ((s + n - 1) / n + kSsmTile - 1) / kSsmTile * kSsmTile;
    const int64_t waves = (blocks * n + sms - 1) / sms, joins = (n + kJoinAhead - 1) / kJoinAhead;
    double cost = static_cast<double>(waves) * static_cast<double>(len + 48);
    if (n > 1) cost = cost * walk + start + static_cast<double>(joins) * join;
    if (n > 1 && cost > 0.97 * least) continue;
    least = cost;
    k.chunk_len = len;
  }
  k.chunks = static_cast<int32_t>((s + k.chunk_len - 1) / k.chunk_len);
  const int64_t parts = b * k.chunks, width = t * c;
  if (k.chunks > 1) {
    k.carry = static_cast<size_t>(parts * width * n);
    k.steps = static_cast<size_t>(parts * width);
  }
  if (bwd) {
    if (k.slabs > 1)
      k.partial_bc = static_cast<size_t>(b * s) * t * groups * k.slabs * 2 * n;
    k.partial_params = static_cast<size_t>(parts * width) * (n + 2);
  }
  return k;
}

cudaError_t launch_ssm_fwd(const SsmParams& p, int dtype, cudaStream_t st) {
  return dtype == SP_BF16  ? launch_states<SP_BF16>(p, st)
         : dtype == SP_F16 ? launch_states<SP_F16>(p, st)
                           : launch_states<SP_F32>(p, st);
}

}  // namespace spb
