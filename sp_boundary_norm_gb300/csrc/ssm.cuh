// Shared parts of the selective state space scan.  Every channel has N states:
//   d = softplus(dt + dt_bias)   (or dt + dt_bias)
//   h[n] = exp(d A[n]) h[n] + d u B[n]
//   y = (sum_n C[n] h[n] + D u) silu(z)
// B and C are shared by a group's channels.
//
// In the walks a lane holds four states (two for N = 8) of two channels side by side, so B
// and C of a token are read from shared memory once for both: a word there costs a warp as
// much as four of its arithmetic instructions.  A channel's lanes put their parts of its
// sums over states into shared memory, where the warps that finish tokens add them up.
#pragma once

#include "region.cuh"

namespace spb {

template <int N>
struct SsmLanes {
  static constexpr int kStates = N >= 16 ? 4 : 2;   // of a channel, in a lane
  static constexpr int kPairs = kStates / 2;
  static constexpr int kLanes = N / kStates;        // of a channel: 4, 4, 8, 16
  static constexpr int kChannels = 2 * 32 / kLanes; // of a warp: 16, 16, 8, 4
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kAll = 0xFFFFFFFFu;

// A lane's states, in memory side by side.
template <int K>
__device__ __forceinline__ void load_states(const float* src, F2 (&h)[K]) {
  if constexpr (K == 2) {
    const float4 v = *reinterpret_cast<const float4*>(src);
    h[0] = f2(v.x, v.y);
    h[1] = f2(v.z, v.w);
  } else {
    const float2 v = *reinterpret_cast<const float2*>(src);
    h[0] = f2(v.x, v.y);
  }
}
template <int K>
__device__ __forceinline__ void store_states(float* dst, const F2 (&h)[K]) {
  const float2 a = split(h[0]);
  if constexpr (K == 2) {
    const float2 b = split(h[1]);
    *reinterpret_cast<float4*>(dst) = make_float4(a.x, a.y, b.x, b.y);
  } else {
    *reinterpret_cast<float2*>(dst) = a;
  }
}
template <int K>
__device__ __forceinline__ void clear(F2 (&h)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) h[k] = 0;
}
// src's states, or zero without one
template <int K>
__device__ __forceinline__ void load_states_or_zero(const float* base, int64_t at, F2 (&h)[K]) {
  if (base != nullptr) load_states(base + at, h);
  else clear(h);
}

// 2^x of both, to about 2^-23 for x <= 0; subnormal results are flushed.
__device__ __forceinline__ F2 pow2(F2 x) {
  float2 v = split(x);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v.y));
  return f2(v.x, v.y);
}

__device__ __forceinline__ float pow2(float x) {
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
  return x;
}

// The same for the decay of a token on its own, to a rounding: near 1 by a polynomial for
// (2^x - 1) / x, fitted to the least relative error over [-1/8, 0] (2^-27).  The power above
// is off to one side there, by 2.5e-8 on the mean at x = -0.01, and a state adds that up over
// all the tokens that it remembers.
__device__ __forceinline__ float decay(float x) {
  float q = fmaf(x, 0.00931570679f, 0.05548395216f);
  q = fmaf(x, q, 0.24022619426f);
  q = fmaf(x, q, kLn2);
  constexpr int kLeast = static_cast<int>(0xBE000000u);      // [-1/8, -0], as integers
  return __float_as_int(x) <= kLeast ? fmaf(x, q, 1.f) : pow2(x);
}
__device__ __forceinline__ F2 decay2(F2 x) {
  const float2 v = split(x);
  return f2(decay(v.x), decay(v.y));
}

// Whole steps' tokens take the power above, and what it loses is made up for once a step:
// `all` is the product of the decays, x the sum of their exponents, and the states behind
// them are multiplied by 2^x / all, as 1 + (2^x - all) (2 - all): slow states by what the
// power has lost, fast ones, which forget it, by nearly 1.  (The polynomial for every token
// makes the same digits: 8 x 8192 x 1024 packed forward 607 us, so 522; without either 467,
// and a state that remembers 1000 tokens off by 1e-5.)  Growing states, and products that
// left float32's range on the way, are left as they are.
// EXACT: for a call's only step.
template <bool EXACT = false>
__device__ __forceinline__ F2 settle2(F2 x, F2 all) {
  const F2 lost = fma2(all, f2(-1.f, -1.f), EXACT ? decay2(x) : pow2(x));
  const F2 inverse = fma2(all, f2(-1.f, -1.f), f2(2.f, 2.f));
  const float2 v = split(x), c = split(mul2(lost, inverse));
  constexpr float kMost = 0x1p-12f;
  return f2(v.x <= 0.5f && fabsf(c.x) <= kMost ? 1.f + c.x : 1.f,
            v.y <= 0.5f && fabsf(c.y) <= kMost ? 1.f + c.y : 1.f);
}

// softplus(x) = max(x, 0) + log(1 + e), e = exp(-|x|), and its derivative
// 1 / (1 + exp(-x)).  log(1 + e) = 2 artanh(s), s = e / (2 + e) <= 1/3, as s times a
// polynomial in s^2 fitted to the least relative error over that range (2^-27): the
// digits of a small e are kept.  e itself is off by 2^-24 |x|, 2^-22 for float32 data.
template <int DT>
__device__ __forceinline__ F2 softplus2(F2 x, F2* slope) {
  const float2 v = split(x);
  F2 e;
  if constexpr (DT == SP_F32) e = exp2_of<SP_F32, false>(f2(-fabsf(v.x), -fabsf(v.y)));
  else e = pow2(f2(fabsf(v.x) * -kLog2e, fabsf(v.y) * -kLog2e));
  const F2 s = mul2(e, rcp2(add2(e, f2(2.f, 2.f)))), q = mul2(s, s);
  F2 p = f2(0.28011987f, 0.28011987f);
  p = fma2(p, q, f2(0.28001806f, 0.28001806f));
  p = fma2(p, q, f2(0.40021527f, 0.40021527f));
  p = fma2(p, q, f2(0.66666418f, 0.66666418f));
  p = fma2(p, q, f2(2.f, 2.f));
  if (slope != nullptr) {
    // 1 / (1 + e), of which a negative x takes e times that
    const F2 w = rcp2(add2(e, f2(1.f, 1.f)));
    const float2 c = split(w), d = split(mul2(e, w));
    *slope = f2(v.x < 0.f ? d.x : c.x, v.y < 0.f ? d.y : c.y);
  }
  return fma2(p, s, held_above(x, 0.f));
}

// Elements in shared memory, as 16-, 8-, 4- or 2-byte accesses.
template <int DT, int N>
__device__ __forceinline__ void lds_pack(Pack<DT, N>& p, const char* src) {
  constexpr int B = Pack<DT, N>::kBytes;
  if constexpr (B >= 16) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) {
      const uint4 v = *(reinterpret_cast<const uint4*>(src) + i);
      p.w[4 * i] = v.x;
      p.w[4 * i + 1] = v.y;
      p.w[4 * i + 2] = v.z;
      p.w[4 * i + 3] = v.w;
    }
  } else if constexpr (B == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    p.w[0] = v.x;
    p.w[1] = v.y;
  } else if constexpr (B == 4) {
    p.w[0] = *reinterpret_cast<const uint32_t*>(src);
  } else {
    p.w[0] = *reinterpret_cast<const unsigned short*>(src);
  }
}

// All of the block's threads; its parts come here from different code.
template <int THREADS>
__device__ __forceinline__ void meet() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// Which of a tile's tokens (at most 32, one a lane) begin a packed sequence.
struct SsmMarks {
  uint32_t starts;
  int seq;               // this lane's token's sequence
};
__device__ __forceinline__ SsmMarks ssm_marks(const SsmParams& P, int64_t tok0, int n_tok) {
  const int lane = threadIdx.x & 31;
  const int64_t tok = tok0 + (lane < n_tok ? lane : n_tok - 1);
  const int j = find_seq(P.cu_seqlens, P.n_seqs, tok);
  const bool start = lane < n_tok && static_cast<int64_t>(__ldg(P.cu_seqlens + j)) == tok;
  return SsmMarks{__ballot_sync(kAll, start), j};
}

// Where a block works: its batch row, chunk, rank, and channels.
template <int CB>
struct SsmPlace {
  int64_t batch, chunk;
  int r, ch0, live;      // rank; first channel (of the rank) and how many
  int group;
  int slab;              // over the ranks and groups
  int64_t tok0, len;     // the chunk's tokens
  __device__ __forceinline__ SsmPlace(const SsmParams& P) {
    const int all = P.t * P.groups * P.slabs;
    const int64_t at = blockIdx.x / all;
    slab = blockIdx.x - static_cast<int>(at) * all;
    batch = at / P.chunks;
    chunk = at - batch * P.chunks;
    const int rg = slab / P.slabs;
    r = rg / P.groups;
    group = rg - r * P.groups;
    const int of_group = P.c / P.groups, first = (slab - rg * P.slabs) * CB;
    ch0 = group * of_group + first;
    live = of_group - first < CB ? of_group - first : CB;
    tok0 = chunk * P.chunk_len;
    len = P.s - tok0 < P.chunk_len ? P.s - tok0 : P.chunk_len;
  }
};

}  // namespace spb
