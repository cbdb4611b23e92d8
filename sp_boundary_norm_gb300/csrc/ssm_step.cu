// Selective scan of a few tokens, as in decoding: bound by reading and writing the
// states once.  A warp takes the same channels of several sequences side by side, with
// their decay rates in registers, and all of the states that it reads are asked for
// before the first is used.
#include "ssm.cuh"

namespace spb {

constexpr int kStepWarps = 8;
constexpr int kStepRows = 4;           // sequences of a warp

template <int DT>
__device__ __forceinline__ float load_one(const char* src) {
  Pack<DT, 1> p;
  float f[1];
  load_pack(p, src);
  unpack(p, f);
  return f[0];
}

template <int DT, int N>
__global__ void __launch_bounds__(32 * kStepWarps)
ssm_step_kernel(const SsmParams P) {
  using L = SsmLanes<N>;
  constexpr int E = ElemSize<DT>::value, K = L::kPairs, G = L::kLanes;
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t warps = static_cast<int64_t>(P.t) * (P.c / L::kChannels);
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kStepWarps + warp;
  const int64_t part = id / warps;
  const int64_t row0 = part * kStepRows;
  if (row0 >= P.b) return;
  const int wc = static_cast<int>(id - part * warps), per_rank = P.c / L::kChannels;
  const int r = wc / per_rank, ch = (wc - r * per_rank) * L::kChannels + lane / G;
  const int n0 = (lane % G) * L::kStates;
  const int64_t state_at = static_cast<int64_t>(ch) * N + n0;
  const int64_t state_step = static_cast<int64_t>(P.c) * N;
  const int64_t chan = static_cast<int64_t>(r) * P.c + ch;
  const int64_t bn = static_cast<int64_t>(ch / (P.c / P.groups)) * N + n0;
  F2 h[kStepRows][K], a2[K];
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    clear(h[i]);
    if (row0 + i < P.b)
      load_states_or_zero(P.h0[r], (row0 + i) * state_step + state_at, h[i]);
  }
  load_states(P.A + chan * N + n0, a2);
#pragma unroll
  for (int p = 0; p < K; ++p) a2[p] = mul2(a2[p], f2(kLog2e, kLog2e));
  const float bias = P.dt_bias != nullptr ? __ldg(P.dt_bias + chan) : 0.f;
  const float skip = P.D != nullptr ? __ldg(P.D + chan) : 0.f;
  for (int64_t tok = 0; tok < P.s; ++tok) {
    float u[kStepRows], d[kStepRows], z[kStepRows];
    Pack<DT, L::kStates> pb[kStepRows], pc[kStepRows];
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
      const int64_t row = ((row0 + i < P.b ? row0 + i : row0)) * P.s + tok;
      u[i] = load_one<DT>(P.u[r] + row * P.ld_u + ch * E);
      d[i] = load_one<DT>(P.dt[r] + row * P.ld_dt + ch * E);
      z[i] = P.gated ? load_one<DT>(P.z[r] + row * P.ld_z + ch * E) : 0.f;
      load_pack(pb[i], P.B[r] + row * P.ld_B + bn * E);
      load_pack(pc[i], P.C[r] + row * P.ld_C + bn * E);
    }
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
      if (row0 + i >= P.b) break;
      float step = d[i] + bias;
      if (P.softplus) step = split(softplus2(f2(step, step), nullptr)).x;
      F2 b[K], c[K];
      unpack_pairs(pb[i], b);
      unpack_pairs(pc[i], c);
      const F2 d2 = f2(step, step), in = f2(step * u[i], step * u[i]);
#pragma unroll
      for (int p = 0; p < K; ++p)
        h[i][p] = fma2(pow2(mul2(d2, a2[p])), h[i][p], mul2(in, b[p]));
      F2 acc = mul2(h[i][0], c[0]);
      if constexpr (K == 2) acc = fma2(h[i][1], c[1], acc);
      const float2 v = split(acc);
      float part_sum[1] = {v.x + v.y};
      sum_over<1, G>(part_sum, lane, 1);
      float y = fmaf(skip, u[i], part_sum[0]);
      if (P.gated) {
        const F2 zz = f2(z[i], z[i]);
        y *= split(mul2(zz, rcp2(add2(exp2_of<DT, false, -1>(zz), f2(1.f, 1.f))))).x;
      }
      if (lane % G == 0) {
        Pack<DT, 1> p;
        const float f[1] = {y};
        pack(p, f);
        store_pack(P.y[r] + ((row0 + i) * P.s + tok) * P.ld_y + ch * E, p);
      }
    }
  }
  if (P.hT[r] != nullptr) {
#pragma unroll
    for (int i = 0; i < kStepRows; ++i)
      if (row0 + i < P.b) store_states(P.hT[r] + (row0 + i) * state_step + state_at, h[i]);
  }
}

template <int DT, int N>
static cudaError_t launch_step(const SsmParams& p, cudaStream_t st) {
  const int64_t warps = static_cast<int64_t>(p.t) * (p.c / SsmLanes<N>::kChannels) *
                        ((p.b + kStepRows - 1) / kStepRows);
  void* args[] = {const_cast<SsmParams*>(&p)};
  return launch_pdl(reinterpret_cast<const void*>(&ssm_step_kernel<DT, N>),
                    dim3(static_cast<unsigned>((warps + kStepWarps - 1) / kStepWarps)),
                    dim3(32 * kStepWarps), 0, args, st);
}

template <int DT>
static cudaError_t launch_states(const SsmParams& p, cudaStream_t st) {
  switch (p.n) {
    case 8: return launch_step<DT, 8>(p, st);
    case 16: return launch_step<DT, 16>(p, st);
    case 32: return launch_step<DT, 32>(p, st);
    default: return launch_step<DT, 64>(p, st);
  }
}

cudaError_t launch_ssm_step(const SsmParams& p, int dtype, cudaStream_t st) {
  return dtype == SP_BF16  ? launch_states<SP_BF16>(p, st)
         : dtype == SP_F16 ? launch_states<SP_F16>(p, st)
                           : launch_states<SP_F32>(p, st);
}

}  // namespace spb
