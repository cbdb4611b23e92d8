// Shared parts of the causal convolution along the tokens, each channel on its own:
//   q[i] = bias + sum_j w[j] x[i - (W - 1) + j],   y[i] = act(q[i])
// where inputs before a sequence's begin come from its state x0 (or are zero).
#pragma once

#include "region.cuh"

namespace spb {

constexpr int kConvThreads = 128;

// Four channels of a token a thread: eight 16-bit ones need half as many registers again
// for weights and windows as leave an SM enough warps.
constexpr int kConvVec = 4;

// The sequence that a thread's run is in: its number (states are found by it), first
// token and end, counted from the run's first token (an end far behind it: anything
// large).
struct ConvSeq {
  int id, lo, hi;
};
template <bool PACKED>
__device__ __forceinline__ ConvSeq conv_seq(const ConvParams& P, int64_t batch, int64_t i0, int i) {
  int64_t lo = 0, hi = P.s;
  int id = static_cast<int>(batch);
  if constexpr (PACKED) {              // in bounds whatever cu holds
    id = find_seq(P.cu_seqlens, P.n_seqs, i0 + i);
    lo = __ldg(P.cu_seqlens + id);
    hi = __ldg(P.cu_seqlens + id + 1);
    lo = lo < 0 ? 0 : lo > i0 + i ? i0 + i : lo;
    hi = hi > P.s || hi <= i0 + i ? P.s : hi;
  }
  return ConvSeq{id, lo < i0 - 8 ? -8 : static_cast<int>(lo - i0),
                 hi > i0 + (1 << 20) ? 1 << 20 : static_cast<int>(hi - i0)};
}

// A lane's taps: for each the weights of its V channels, and its bias.
template <int DT, int V, int W>
struct Taps {
  F2 w[W][V / 2], bias[V / 2];
  __device__ __forceinline__ void load(const ConvParams& P, int64_t ch) {
    constexpr int E = ElemSize<DT>::value;
    float f[V * W];
    Pack<DT, V * W> p;
    constexpr int kPieces = sizeof(p.w) / 8;        // 8-byte pieces: V * W * E is a multiple
    const char* src = P.weight + ch * W * E;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(src) + i);
      p.w[2 * i] = v.x;
      p.w[2 * i + 1] = v.y;
    }
    unpack(p, f);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int k = 0; k < V / 2; ++k) w[j][k] = f2(f[2 * k * W + j], f[(2 * k + 1) * W + j]);
    Pack<DT, V> q{};
    if (P.bias != nullptr) load_pack(q, P.bias + ch * E);
    unpack_pairs(q, bias);
  }
  // bias + the taps on the window (oldest first) and the token itself
  __device__ __forceinline__ void apply(const F2 (&win)[W - 1][V / 2], const F2 (&x)[V / 2],
                                        F2 (&q)[V / 2]) const {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      F2 a = bias[k];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) a = fma2(w[j][k], win[j][k], a);
      q[k] = fma2(w[W - 1][k], x[k], a);
    }
  }
};

// Forgets the oldest row, takes x as the newest.
template <int W, int K>
__device__ __forceinline__ void shift(F2 (&win)[W - 1][K], const F2 (&x)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j) win[j][k] = win[j + 1][k];
    win[W - 2][k] = x[k];
  }
}

// The W - 1 inputs before the run's token i, in sequence q; x: the run's first token, x0:
// the call's first state (or NULL), both at this lane's channels.
template <int DT, int V, int W>
__device__ __forceinline__ void load_window(const ConvParams& P, const char* x, const char* x0,
                                            const ConvSeq& q, int i, F2 (&win)[W - 1][V / 2]) {
  constexpr int E = ElemSize<DT>::value;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int row = i - (W - 1) + j;
    Pack<DT, V> p{};
    if (row >= q.lo) {
      load_pack(p, x + row * P.ld_x);
    } else if (x0 != nullptr) {
      load_pack(p, x0 + (static_cast<int64_t>(q.id) * (W - 1) + (W - 1 + row - q.lo)) * P.c * E);
    }
    unpack_pairs(p, win[j]);
  }
}

// Rows on their way to a thread: its own pieces of shared memory, a group of rows after
// another, kConvAhead groups asked for before the first is used.  They take no registers
// and no barrier.
constexpr int kConvGroup = 4, kConvAhead = 2;
template <int DT, int V, int TENSORS>
struct RowRing {
  static constexpr int kBytes = V * ElemSize<DT>::value;
  static constexpr int kGroups = kConvAhead + 1;
  static constexpr int kSize = kGroups * kConvGroup * TENSORS * kConvThreads * kBytes;
  char* mine;
  const char* src[TENSORS];
  int64_t ld[TENSORS];
  int put = 0, get = 0;                // groups' places, in bytes
  static constexpr int kStep = kConvGroup * TENSORS * kConvThreads * kBytes;
  __device__ __forceinline__ explicit RowRing(char* smem) : mine(smem + threadIdx.x * kBytes) {}
  // asks for the next group's first `rows` rows
  __device__ __forceinline__ void ask(int rows) {
    if (rows >= kConvGroup) {
#pragma unroll
      for (int u = 0; u < kConvGroup; ++u) ask_row(u);
    } else {
#pragma unroll 1
      for (int u = 0; u < rows; ++u) ask_row(u);
    }
    cp_async_commit();
    put = put == (kGroups - 1) * kStep ? 0 : put + kStep;
  }
  __device__ __forceinline__ void ask_row(int u) {
#pragma unroll
    for (int t = 0; t < TENSORS; ++t) {
      char* dst = mine + put + (u * TENSORS + t) * kConvThreads * kBytes;
      if constexpr (kBytes == 16) cp_async16(dst, src[t]);
      else cp_async8(dst, src[t]);
      src[t] += ld[t];
    }
  }
  __device__ __forceinline__ void row(int u, int t, Pack<DT, V>& p) const {
    const char* from = mine + get + (u * TENSORS + t) * kConvThreads * kBytes;
    if constexpr (kBytes == 16) {
      const uint4 v = lds16(from);
      p.w[0] = v.x;
      p.w[1] = v.y;
      p.w[2] = v.z;
      p.w[3] = v.w;
    } else {
      const uint2 v = lds8(from);
      p.w[0] = v.x;
      p.w[1] = v.y;
    }
  }
  __device__ __forceinline__ void next() {
    get = get == (kGroups - 1) * kStep ? 0 : get + kStep;
  }
};

}  // namespace spb
