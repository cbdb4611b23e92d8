// Shared parts of the gated recurrence's forward and backward:
//   a = sigmoid(gate), k = 1 - a = sigmoid(-gate)
//   h[i] = a[i] h[i-1] + k[i] v[i]   (tied)   or   a[i] h[i-1] + v[i]   (free)
// along the tokens of a sequence, each channel on its own.
//
// A block takes 64 channels, two a lane, and 16 tokens a warp (a "run"): lane
// and warp read whole 128-byte row pieces, a thread scans its run in registers
// and knows it as an affine map h -> A h + H.  The maps are joined over the
// block's warps in shared memory and over the blocks of a cluster by
// distributed shared memory, always in token order, so results do not depend
// on timing; then the cluster steps to the next stretch of the sequence with
// the state in registers.  Nothing is read twice and no block waits for
// another but its cluster's.
#pragma once

#include "region.cuh"

namespace spb {

// Two channels of one token.
template <int DT>
using Two = Pack<DT, 2>;

// sigmoid(g) and sigmoid(-g), each with a small relative error: with
// e = exp(g), k = 1 / (1 + e) and a = e k.  The exponent is capped where k is
// the smallest normal float (exp would overflow); NaN stays NaN.
template <int DT>
__device__ __forceinline__ void gate_of(float g, float& a, float& k) {
  float e;
  if constexpr (DT == SP_F32) {
    asm("min.NaN.f32 %0, %1, 0f42AE0000;" : "=f"(g) : "f"(g));   // 87
    e = expf(g);
    k = __frcp_rn(1.f + e);
  } else {
    // 16-bit gates: the fast exponential's error (a few 1e-7) is far below
    // the rounding of the outputs
    asm("min.NaN.f32 %0, %1, 0f42FC0000;" : "=f"(g) : "f"(g * 1.4426950408889634f));   // 126
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(k) : "f"(1.f + e));
  }
  a = e * k;
}

// The affine maps of a thread's two channels over some tokens.
struct alignas(16) Map2 {
  float a0, a1, h0, h1;
};

// later(earlier(h)) of one channel.  A sequence that begins inside the later
// part cuts the earlier one off: its factor is exactly zero, and what the
// earlier part holds (an infinity, a NaN) must not pass.
template <bool PACKED>
__device__ __forceinline__ float through(float a, float h, float x) {
  return PACKED && a == 0.f ? h : fmaf(a, x, h);
}

__device__ __forceinline__ void st_cluster_map(uint32_t cluster_addr, const Map2& m) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "f"(m.a0),
               "f"(m.a1), "f"(m.h0), "f"(m.h1)
               : "memory");
}

// Which of the run's tokens tok0 .. tok0 + 15 begin a sequence, and which end one.
struct RunMarks {
  uint32_t starts, ends;
};

template <bool PACKED>
__device__ __forceinline__ RunMarks run_marks(const ScanParams& P, int64_t tok0) {
  if (tok0 >= P.s) return RunMarks{0u, 0u};
  // bit i: token tok0 + i is the first of a sequence, or the first after the call's last
  uint32_t m = tok0 == 0 ? 1u : 0u;
  if constexpr (PACKED) {
    const int64_t end = tok0 + kScanRun < P.s - 1 ? tok0 + kScanRun : P.s - 1;
    const int lane = threadIdx.x & 31;
    for (int j = seq_of_token(P.cu_seqlens, P.n_seqs, tok0); j < P.n_seqs; j += 32) {
      const int64_t at = j + lane < P.n_seqs ? __ldg(P.cu_seqlens + j + lane) : end + 1;
      const bool in = at >= tok0 && at <= end;
      m |= __reduce_or_sync(0xFFFFFFFFu, in ? 1u << static_cast<int>(at - tok0) : 0u);
      if (__any_sync(0xFFFFFFFFu, at > end)) break;
    }
  }
  const int left = P.s - tok0 <= kScanRun ? static_cast<int>(P.s - tok0) : kScanRun + 1;
  const uint32_t starts = m & ((1u << (left < kScanRun ? left : kScanRun)) - 1u);
  if (left <= kScanRun) m |= 1u << left;
  return RunMarks{starts, (m >> 1) & 0xFFFFu};
}

template <bool PACKED>
__device__ __forceinline__ int seq_at(const ScanParams& P, int bi, int64_t tok) {
  if constexpr (PACKED) return seq_of_token(P.cu_seqlens, P.n_seqs, tok);
  return bi;
}

// The two channels' values of each marked token's sequence, from `src`
// (float32 [sequences][c], NULL = zeros) into the thread's slots.
template <bool PACKED>
__device__ __forceinline__ void fetch_states(const ScanParams& P, const float* src, uint32_t marks,
                                             int64_t tok0, int bi, int ch, bool on,
                                             float2 (*slot)[32]) {
  const int lane = threadIdx.x & 31;
  while (marks != 0) {
    const int i = __ffs(marks) - 1;
    marks &= marks - 1;
    float2 v = make_float2(0.f, 0.f);
    if (src != nullptr) {
      const int seq = seq_at<PACKED>(P, bi, tok0 + i);
      if (on)
        v = *reinterpret_cast<const float2*>(src + static_cast<int64_t>(seq) * P.c + ch);
    }
    slot[i][lane] = v;
  }
}

// The reverse: the slots of the marked tokens to their sequences in `dst`.
template <bool PACKED>
__device__ __forceinline__ void put_states(const ScanParams& P, float* dst, uint32_t marks,
                                           int64_t tok0, int bi, int ch, bool on,
                                           float2 (*slot)[32]) {
  const int lane = threadIdx.x & 31;
  while (marks != 0) {
    const int i = __ffs(marks) - 1;
    marks &= marks - 1;
    const int seq = seq_at<PACKED>(P, bi, tok0 + i);
    if (on)
      *reinterpret_cast<float2*>(dst + static_cast<int64_t>(seq) * P.c + ch) = slot[i][lane];
  }
}

// A sequence without tokens passes its state (or its gradient) on.  By one
// block of the unit, 64 channels, whole warps over the sequences.
__device__ __forceinline__ void pass_empty(const ScanParams& P, const float* src, float* dst,
                                           int ch, bool on) {
  if (dst == nullptr || dst == src) return;
  for (int j = threadIdx.x >> 5; j < P.n_seqs; j += blockDim.x >> 5) {
    if (__ldg(P.cu_seqlens + j) != __ldg(P.cu_seqlens + j + 1) || !on) continue;
    const int64_t at = static_cast<int64_t>(j) * P.c + ch;
    *reinterpret_cast<float2*>(dst + at) =
        src != nullptr ? *reinterpret_cast<const float2*>(src + at) : make_float2(0.f, 0.f);
  }
}

// Joins the runs' maps in token order (TIME = +1) or against it (-1).  `mine`:
// this thread's run; returns the value entering it, from the value `carry`
// that enters the cluster's stretch, and moves `carry` behind the stretch.
// One block barrier and one cluster barrier; the buffers alternate, so the
// next call writes the other pair.
struct ScanShared {
  Map2 run[2][kScanMaxWarps][32];
  Map2 block[2][kScanMaxCluster][32];
};

template <bool PACKED, int TIME>
__device__ __forceinline__ float2 join_runs(ScanShared& sh, int par, const Map2& mine, int C,
                                            int rank, float2& carry) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  sh.run[par][warp][lane] = mine;
  __syncthreads();
  float2 in = carry;
  if (C > 1) {
    if (warp < C) {
      Map2 b = sh.run[par][TIME > 0 ? 0 : nw - 1][lane];
      for (int k = 1; k < nw; ++k) {
        const Map2 m = sh.run[par][TIME > 0 ? k : nw - 1 - k][lane];
        b.h0 = through<PACKED>(m.a0, m.h0, b.h0);
        b.h1 = through<PACKED>(m.a1, m.h1, b.h1);
        b.a0 = through<PACKED>(m.a0, 0.f, b.a0);
        b.a1 = through<PACKED>(m.a1, 0.f, b.a1);
      }
      for (int peer = warp; peer < C; peer += nw)
        st_cluster_map(cluster_map(&sh.block[par][rank][lane], peer), b);
    }
    cluster_sync_all();
    float2 x = carry;
    for (int k = 0; k < C; ++k) {
      const int r = TIME > 0 ? k : C - 1 - k;
      if (r == rank) in = x;
      const Map2 m = sh.block[par][r][lane];
      x.x = through<PACKED>(m.a0, m.h0, x.x);
      x.y = through<PACKED>(m.a1, m.h1, x.y);
    }
    carry = x;
  }
  float2 x = in, got = in;
  const int upto = C > 1 ? (TIME > 0 ? warp : nw - 1 - warp) : nw;
  for (int k = 0; k < upto; ++k) {
    const int w = TIME > 0 ? k : nw - 1 - k;
    if (w == warp) got = x;
    const Map2 m = sh.run[par][w][lane];
    x.x = through<PACKED>(m.a0, m.h0, x.x);
    x.y = through<PACKED>(m.a1, m.h1, x.y);
  }
  if (C > 1) return x;
  carry = x;
  return got;
}

// Launches a scan kernel: `warps` warps a block, p.cluster blocks a cluster.
cudaError_t launch_scan(const void* fn, const ScanParams& p, int warps, void** args,
                        cudaStream_t st);

}  // namespace spb
