// Selective scan of a few tokens of many sequences, as in decoding: bound by reading and
// writing the states once.  A block takes the channels of eight warps and walks sequences,
// as many a step as have 16 tokens (at most four).  A step's states and tokens are asked
// for one step ahead; the tokens are prepared (softplus, d u, D u, silu(z)) once for each
// channel in shared memory, where a channel's lanes then find them.  Measured on a GB300,
// bf16, 64 sequences of 8 ranks' 1024 channels of 16 states: 72 MB in 18.3 us, 3.9 TB/s; with
// the hardware's power alone for a decay 17.7, as the same accesses without the arithmetic.
// (A block for every sequence and 32 channels, which prepared its tokens itself: 23 us; three
// blocks an SM 21.)
//
// Up to 16 tokens a sequence (kSsmStepTokens) come here.  The other form's blocks start up
// for one sequence each: 64 sequences of 1, 4, 8 and 16 tokens took 15, 33, 53 and 95 us
// here (in place, replayed) and 123, 138, 160 and 165 there; one sequence of 1, 8 and 16
// tokens 2.3, 3.1 and 4.1 here and 3.1, 3.7 and 3.5 there.
#include "ssm.cuh"

namespace spb {

constexpr int kStepThreads = 256;
constexpr int kStepBlocks = 4;         // of an SM, by their registers

// The sum over a channel's L lanes, in a fixed order.
template <int L>
__device__ __forceinline__ float over_lanes(float v) {
#pragma unroll
  for (int step = L / 2; step > 0; step /= 2) v += __shfl_xor_sync(kAll, v, step);
  return v;
}

// R: sequences of a step, with kSsmStepTokens tokens in all at most
template <int DT, int N, int R>
__global__ void __launch_bounds__(kStepThreads, kStepBlocks)
ssm_step_kernel(const SsmParams P) {
  using L = SsmLanes<N>;
  constexpr int E = ElemSize<DT>::value, K = L::kPairs, G = L::kLanes;
  constexpr int CB = kStepThreads / G;
  // Up to four tokens have exact decays each; of more, the call's are made up for together
  // (64 sequences of 16 tokens 95 us, so 109, without either 82; of four 32, so 33).
  constexpr bool kSettled = R < 4;
  __shared__ float4 prepared[2][kSsmStepTokens][CB];       // d, d u, D u, silu(z)
  __shared__ __align__(16) float shared[2][kSsmStepTokens][2 * N];
  pdl_wait();
  const int tid = threadIdx.x;
  const int per_part = P.t * P.groups * P.slabs;
  const int part = blockIdx.x / per_part, slab = blockIdx.x - part * per_part;
  const int rg = slab / P.slabs;
  const int r = rg / P.groups, group = rg - r * P.groups;
  const int of_group = P.c / P.groups, first = (slab - rg * P.slabs) * CB;
  const int ch0 = group * of_group + first;
  const int live = of_group - first < CB ? of_group - first : CB;
  // the block's sequences: chunk_len of them a part
  const int row0 = part * static_cast<int>(P.chunk_len);
  const int rows = P.b - row0 < P.chunk_len ? P.b - row0 : static_cast<int>(P.chunk_len);
  const int s = static_cast<int>(P.s);

  const bool on = tid / G < live;
  const int ch = ch0 + (on ? tid / G : 0), n0 = (tid % G) * L::kStates;
  const int64_t chan = static_cast<int64_t>(r) * P.c;
  const int64_t state_step = static_cast<int64_t>(P.c) * N;
  const int64_t state_at = row0 * state_step + static_cast<int64_t>(ch) * N + n0;
  const float* h0 = P.h0[r] != nullptr && on ? P.h0[r] + state_at : nullptr;
  float* hT = P.hT[r] != nullptr && on ? P.hT[r] + state_at : nullptr;
  F2 a2[K];
  load_states(P.A + (chan + ch) * N + n0, a2);
#pragma unroll
  for (int p = 0; p < K; ++p) a2[p] = mul2(a2[p], f2(kLog2e, kLog2e));

  // What a thread asks for of the next step: its states, two channels of a token, and four
  // values of B or C (threads from the last one on).
  F2 next[R][K];
  Pack<DT, 2> pu, pd, pz;
  Pack<DT, 4> pbc;
  auto read_pair = [&](int64_t row, int c) {
    load_pack(pu, P.u[r] + row * P.ld_u + (ch0 + c) * E);
    load_pack(pd, P.dt[r] + row * P.ld_dt + (ch0 + c) * E);
    if (P.gated) load_pack(pz, P.z[r] + row * P.ld_z + (ch0 + c) * E);
  };
  auto read_shared = [&](int64_t row, int e) {
    const int64_t n = (e % N + group * N) * E;
    if (e < N) load_pack(pbc, P.B[r] + row * P.ld_B + n);
    else load_pack(pbc, P.C[r] + row * P.ld_C + n);
  };
  constexpr int kHalf = CB / 2, kQuads = N / 2;
  const int my_c = tid % kHalf * 2, my_k = tid / kHalf;
  const int my_e = (kStepThreads - 1 - tid) % kQuads * 4, my_q = (kStepThreads - 1 - tid) / kQuads;
  auto ask = [&](int i0) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      clear(next[i]);
      if (h0 != nullptr && i0 + i < rows) load_states(h0 + i * state_step, next[i]);
    }
    if (h0 != nullptr) h0 += R * state_step;
    const int tokens = (rows - i0 < R ? rows - i0 : R) * s;
    const int64_t row = static_cast<int64_t>(row0 + i0) * s;
    if (my_k < tokens && my_c < live) read_pair(row + my_k, my_c);
    if (my_q < tokens) read_shared(row + my_q, my_e);
  };
  auto prepare = [&](int i0, int buffer) {
    const int tokens = (rows - i0 < R ? rows - i0 : R) * s;
    const int64_t row = static_cast<int64_t>(row0 + i0) * s;
    for (int k = my_k; k < tokens && my_c < live; k += kStepThreads / kHalf) {
      if (k != my_k) read_pair(row + k, my_c);
      F2 u[1], d[1], z[1], bias = 0, skip = 0;
      if (P.dt_bias != nullptr) bias = *reinterpret_cast<const F2*>(P.dt_bias + chan + ch0 + my_c);
      if (P.D != nullptr) skip = *reinterpret_cast<const F2*>(P.D + chan + ch0 + my_c);
      unpack_pairs(pu, u);
      unpack_pairs(pd, d);
      unpack_pairs(pz, z);
      F2 step = add2(d[0], bias);
      if (P.softplus) step = softplus2<DT>(step, nullptr);
      const F2 gate = P.gated ? mul2(z[0], rcp2(add2(exp2_of<DT, false, -1>(z[0]), f2(1.f, 1.f))))
                              : f2(1.f, 1.f);
      const float2 a = split(step), b = split(mul2(step, u[0])), e = split(mul2(skip, u[0])),
                   g = split(gate);
      prepared[buffer][k][my_c] = make_float4(a.x, b.x, e.x, g.x);
      prepared[buffer][k][my_c + 1] = make_float4(a.y, b.y, e.y, g.y);
    }
    for (int k = my_q; k < tokens; k += kStepThreads / kQuads) {
      if (k != my_q) read_shared(row + k, my_e);
      float f[4];
      unpack(pbc, f);
      *reinterpret_cast<float4*>(&shared[buffer][k][my_e]) = make_float4(f[0], f[1], f[2], f[3]);
    }
  };
  ask(0);
  prepare(0, 0);
  char* y = P.y[r] + static_cast<int64_t>(row0) * s * P.ld_y + ch * E;
  int buffer = 0;
  for (int i0 = 0; i0 < rows; i0 += R, buffer ^= 1) {
    F2 h[R][K];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int p = 0; p < K; ++p) h[i][p] = next[i][p];
    __syncthreads();                   // the step is prepared, and the one before done with
    if (i0 + R < rows) ask(i0 + R);
    const float4* token = &prepared[buffer][0][tid / G];
    const float* bc = &shared[buffer][0][n0];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i0 + i >= rows) break;
      F2 all[K], steps = 0;
#pragma unroll
      for (int p = 0; p < K; ++p) all[p] = f2(1.f, 1.f);
      for (int t = 0; t < s; ++t, token += CB, bc += 2 * N, y += P.ld_y) {
        const float4 x = *token;
        const F2 step = f2(x.x, x.x), in = f2(x.y, x.y);
        F2 b[K], c[K];
        load_states(bc, b);
        load_states(bc + N, c);
#pragma unroll
        for (int p = 0; p < K; ++p) {
          const F2 e = mul2(step, a2[p]), a = kSettled ? pow2(e) : decay2(e);
          if constexpr (kSettled) all[p] = mul2(all[p], a);
          h[i][p] = fma2(a, h[i][p], mul2(in, b[p]));
        }
        if constexpr (kSettled) steps = add2(steps, step);
        F2 acc = mul2(h[i][0], c[0]);
        if constexpr (K == 2) acc = fma2(h[i][1], c[1], acc);
        const float2 v = split(acc);
        const float sum = over_lanes<G>(v.x + v.y);
        if (on && tid % G == 0) {
          Pack<DT, 1> p;
          const float f[1] = {(sum + x.z) * x.w};
          pack(p, f);
          store_pack(y, p);
        }
      }
      if constexpr (kSettled) {
#pragma unroll
        for (int p = 0; p < K; ++p)
          h[i][p] = mul2(h[i][p], settle2<true>(mul2(steps, a2[p]), all[p]));
      }
      if (hT != nullptr) {
        store_states(hT, h[i]);
        hT += state_step;
      }
    }
    if (i0 + R < rows) prepare(i0 + R, buffer ^ 1);
  }
}

template <int DT, int N, int R>
static cudaError_t launch_step(const SsmParams& p, cudaStream_t st) {
  constexpr int CB = kStepThreads / SsmLanes<N>::kLanes;
  SsmParams q = p;
  q.slabs = (p.c / p.groups + CB - 1) / CB;
  // one wave of blocks, each with as many whole steps of the sequences
  const int64_t across = static_cast<int64_t>(p.t) * p.groups * q.slabs;
  const int64_t steps = (p.b + R - 1) / R;
  int64_t parts = static_cast<int64_t>(device_sm_count()) * kStepBlocks / across;
  parts = parts < 1 ? 1 : parts < steps ? parts : steps;
  q.chunk_len = (steps + parts - 1) / parts * R;
  parts = (p.b + q.chunk_len - 1) / q.chunk_len;
  void* args[] = {&q};
  return launch_pdl(reinterpret_cast<const void*>(&ssm_step_kernel<DT, N, R>),
                    dim3(static_cast<unsigned>(parts * across)), dim3(kStepThreads), 0, args, st);
}

template <int DT, int N>
static cudaError_t launch_rows(const SsmParams& p, cudaStream_t st) {
  return p.s * 4 <= kSsmStepTokens   ? launch_step<DT, N, 4>(p, st)
         : p.s * 2 <= kSsmStepTokens ? launch_step<DT, N, 2>(p, st)
                                     : launch_step<DT, N, 1>(p, st);
}

template <int DT>
static cudaError_t launch_states(const SsmParams& p, cudaStream_t st) {
  switch (p.n) {
    case 8: return launch_rows<DT, 8>(p, st);
    case 16: return launch_rows<DT, 16>(p, st);
    case 32: return launch_rows<DT, 32>(p, st);
    default: return launch_rows<DT, 64>(p, st);
  }
}

cudaError_t launch_ssm_step(const SsmParams& p, int dtype, cudaStream_t st) {
  return dtype == SP_BF16  ? launch_states<SP_BF16>(p, st)
         : dtype == SP_F16 ? launch_states<SP_F16>(p, st)
                           : launch_states<SP_F32>(p, st);
}

}  // namespace spb
