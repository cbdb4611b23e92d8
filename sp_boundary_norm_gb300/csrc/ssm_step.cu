// Selective scan of a few tokens, as in decoding: bound by reading and writing the
// states once.  A block takes the channels of eight warps of four sequences.  All of
// its states are asked for first; while they are on their way the block prepares the
// tokens (softplus, d u, D u, silu(z)) once for each channel in shared memory, where a
// channel's lanes then find them.  Measured on a GB300, bf16, 64 sequences of 8 ranks'
// 1024 channels of 16 states: SSM_STEP_FIGURE.
#include "ssm.cuh"

namespace spb {

constexpr int kStepThreads = 256;
constexpr int kStepRows = 4;           // sequences of a block

template <int DT, int N>
__global__ void __launch_bounds__(kStepThreads)
ssm_step_kernel(const SsmParams P) {
  using L = SsmLanes<N>;
  constexpr int E = ElemSize<DT>::value, K = L::kPairs, G = L::kLanes, R = kStepRows;
  constexpr int CB = kStepThreads / G;
  __shared__ float4 prepared[R * kSsmStepTokens][CB];          // d, d u, D u, silu(z)
  __shared__ __align__(16) float shared[R * kSsmStepTokens][2 * N];
  pdl_wait();
  const int tid = threadIdx.x;
  const int per_row = P.t * P.groups * P.slabs;
  const int64_t part = blockIdx.x / per_row;
  const int slab = blockIdx.x - static_cast<int>(part) * per_row, rg = slab / P.slabs;
  const int r = rg / P.groups, group = rg - r * P.groups;
  const int of_group = P.c / P.groups, first = (slab - rg * P.slabs) * CB;
  const int ch0 = group * of_group + first;
  const int live = of_group - first < CB ? of_group - first : CB;
  const int64_t row0 = part * R;
  const int rows = P.b - row0 < R ? static_cast<int>(P.b - row0) : R;
  const int s = static_cast<int>(P.s);

  const bool on = tid / G < live;
  const int ch = ch0 + (on ? tid / G : 0), n0 = (tid % G) * L::kStates;
  const int64_t chan = static_cast<int64_t>(r) * P.c;
  const int64_t state_step = static_cast<int64_t>(P.c) * N;
  const int64_t state_at = row0 * state_step + static_cast<int64_t>(ch) * N + n0;
  F2 h[R][K], a2[K];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    clear(h[i]);
    if (on && i < rows) load_states_or_zero(P.h0[r], state_at + i * state_step, h[i]);
  }
  load_states(P.A + (chan + ch) * N + n0, a2);

  const int tokens = rows * s;
  for (int i = tid; i < tokens * (CB / 2); i += kStepThreads) {
    const int k = i / (CB / 2), c = (i - k * (CB / 2)) * 2;
    if (c >= live) continue;
    const int64_t row = row0 * s + k;
    Pack<DT, 2> pu, pd, pz{};
    load_pack(pu, P.u[r] + row * P.ld_u + (ch0 + c) * E);
    load_pack(pd, P.dt[r] + row * P.ld_dt + (ch0 + c) * E);
    if (P.gated) load_pack(pz, P.z[r] + row * P.ld_z + (ch0 + c) * E);
    F2 u[1], d[1], z[1], bias = 0, skip = 0;
    if (P.dt_bias != nullptr) bias = *reinterpret_cast<const F2*>(P.dt_bias + chan + ch0 + c);
    if (P.D != nullptr) skip = *reinterpret_cast<const F2*>(P.D + chan + ch0 + c);
    unpack_pairs(pu, u);
    unpack_pairs(pd, d);
    unpack_pairs(pz, z);
    F2 step = add2(d[0], bias);
    if (P.softplus) step = softplus2<DT>(step, nullptr);
    const F2 gate = P.gated ? mul2(z[0], rcp2(add2(exp2_of<DT, false, -1>(z[0]), f2(1.f, 1.f))))
                            : f2(1.f, 1.f);
    const float2 a = split(step), b = split(mul2(step, u[0])), e = split(mul2(skip, u[0])),
                 g = split(gate);
    prepared[k][c] = make_float4(a.x, b.x, e.x, g.x);
    prepared[k][c + 1] = make_float4(a.y, b.y, e.y, g.y);
  }
  for (int i = tid; i < tokens * (N / 2); i += kStepThreads) {
    const int k = i / (N / 2), e = (i - k * (N / 2)) * 4;
    const int64_t row = row0 * s + k, n = e % N + group * N;
    Pack<DT, 4> p;
    float f[4];
    if (e < N) load_pack(p, P.B[r] + row * P.ld_B + n * E);
    else load_pack(p, P.C[r] + row * P.ld_C + n * E);
    unpack(p, f);
    *reinterpret_cast<float4*>(&shared[k][e]) = make_float4(f[0], f[1], f[2], f[3]);
  }
#pragma unroll
  for (int p = 0; p < K; ++p) a2[p] = mul2(a2[p], f2(kLog2e, kLog2e));
  __syncthreads();

#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i >= rows) break;
    for (int tok = 0; tok < s; ++tok) {
      const int k = i * s + tok;
      const float4 x = prepared[k][tid / G];
      const F2 step = f2(x.x, x.x), in = f2(x.y, x.y);
      F2 b[K], c[K];
      load_states(&shared[k][n0], b);
      load_states(&shared[k][N + n0], c);
#pragma unroll
      for (int p = 0; p < K; ++p)
        h[i][p] = fma2(pow2(mul2(step, a2[p])), h[i][p], mul2(in, b[p]));
      F2 acc = mul2(h[i][0], c[0]);
      if constexpr (K == 2) acc = fma2(h[i][1], c[1], acc);
      const float2 v = split(acc);
      float sum[1] = {v.x + v.y};
      sum_over<1, G>(sum, tid, 1);
      if (on && tid % G == 0) {
        Pack<DT, 1> p;
        const float f[1] = {(sum[0] + x.z) * x.w};
        pack(p, f);
        store_pack(P.y[r] + (row0 * s + k) * P.ld_y + ch * E, p);
      }
    }
    if (on && P.hT[r] != nullptr) store_states(P.hT[r] + state_at + i * state_step, h[i]);
  }
}

template <int DT, int N>
static cudaError_t launch_step(const SsmParams& p, cudaStream_t st) {
  constexpr int CB = kStepThreads / SsmLanes<N>::kLanes;
  SsmParams q = p;
  q.slabs = (p.c / p.groups + CB - 1) / CB;
  const int64_t grid = static_cast<int64_t>((p.b + kStepRows - 1) / kStepRows) * p.t * p.groups *
                       q.slabs;
  void* args[] = {&q};
  return launch_pdl(reinterpret_cast<const void*>(&ssm_step_kernel<DT, N>),
                    dim3(static_cast<unsigned>(grid)), dim3(kStepThreads), 0, args, st);
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
