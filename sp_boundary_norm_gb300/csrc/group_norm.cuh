// Shared parts of group norm with an activation, channels last:
//   z = (x - mean) rstd over the l rows and c / groups channels of a group of
//   one sample,  q = z gamma + beta,  y = q or q sigmoid(q).
//
// A thread owns one vector of 8 channels (its column; all of one group) and
// walks rows, so the parameters and their gradients stay in registers.  Four
// forms, by the size of a sample:
//  - rows: samples of one row (the per-token norm of heads); a warp, or for wide
//    groups the warps of a group, takes whole groups of several rows at once;
//  - tiles: a block takes several whole samples of few rows; every thread holds
//    its vectors in registers between the statistics and the result;
//  - held: a small block takes one sample's slab of groups at a time, as many
//    vectors a thread as its registers hold;
//  - units: a cluster of blocks takes one sample's slab of groups, reads it for
//    the statistics, joins them through distributed shared memory, and reads it
//    again, from L2 as far as the clusters at work fit it, for the result.  (Kept
//    in shared memory instead, the slab left so few warps an SM that the
//    arithmetic took longer than the second reading: 8 samples of 4096 x 1280
//    in 48 us forward and 90 backward, persistent blocks with the next sample's
//    copies beneath the stores 57 and 107.)
// Measured on a GB300, bf16, LayerNorm and SiLU, forward and backward (the floor
// is the time of x, y and dy, dx at the measured copy rate, 6.8 TB/s):
//   rows: 16,384 of 8 ranks' 8 groups of 128, RMS 93 and 159 us (floor 79, 119),
//     bound by the arithmetic's latency at two blocks an SM, two thirds of the
//     issue slots taken;
//   tiles: 16,384 samples of 4 rows of 512 50 and 61 (20, 30), bound by the
//     barriers around each tile's sums;
//   held: 1365 samples of 48 rows of 512 39 and 72 (20, 30), bound by the time from
//     a sample's loads to its stores;
//   units: 8 samples of 4096 x 1280 45 and 80 (25, 37): the second reading, from
//     L2, and the joins add what is above the floor.
// Sums run in a fixed order: results do not depend on timing.  Statistics are
// two-pass (of values held in registers) and joined as (count, mean, M2), so a
// mean far above the spread costs no digits.
#pragma once

#include "region.cuh"

namespace spb {

template <int DT>
using Vec8 = Pack<DT, 8>;

constexpr int kTileRows = 4;        // vectors a thread holds (tiles; forward)
constexpr int kBackTileRows = 2;    // of x and of dy (tiles; backward)
// Vectors of x a thread holds in the rows form, and blocks an SM that the
// registers are held to (16,384 rows of 8 x 1024, RMS, of an earlier state of the
// kernel: 4 and 2 95 us, 2 and 4 93, 2 and 3 97, 4 and 3 116 with spilled registers;
// wider groups and odd ones want the four; float32 2 and 3 95 us, 4 and 2 111).
template <int DT>
constexpr int kRowRows = DT == SP_F32 ? 2 : 4;
template <int DT>
constexpr int kRowBlocks = DT == SP_F32 ? 3 : 2;
constexpr int kBackRowRows = 2;     // of x and of dy, with two blocks an SM
constexpr int kBackRowBlocks = 2;
constexpr int kRowWarps = 8;        // of a block (rows), more for groups beyond 256 vectors
constexpr int kRowMaxWarps = kGroupThreads / 32;

// Units: blocks an SM that the registers are held to, and vectors on their way to
// a thread, in the backward of x and of dy each (8 samples of 4096 x 1280: forward,
// 3 and 6 45 us, 2 and 4 49; backward, 2 and 4 78).
constexpr int kUnitBlocks = 3, kBackUnitBlocks = 2;
template <int DT>
constexpr int kUnitRing = DT == SP_F32 ? 3 : 6;
template <int DT>
constexpr int kWideRing = DT == SP_F32 ? 4 : 8;
template <int DT>
constexpr int kBackUnitRing = DT == SP_F32 ? 2 : 4;

// Held: vectors a thread keeps (forward), and of x and dy each (backward), and
// blocks of 256 threads an SM that the registers are held to.
constexpr int kHeldBlocks = 2;
template <int DT>
constexpr int kHold = DT == SP_F32 ? 6 : 12;
template <int DT>
constexpr int kBackHold = DT == SP_F32 ? 3 : 6;

// How the lanes of a group add up (rows form): a power of two of neighbouring
// lanes by shuffles; other widths up to 31 through the warp's shared memory,
// every lane adding its group's values; wider groups in their warps, then over
// the warps (a team) through shared memory.
constexpr int kSumLanes = 0, kSumWarp = 1, kSumTeam = 2;

__device__ __forceinline__ F2 both(float v) { return f2(v, v); }

template <int DT>
__device__ __forceinline__ F2 sigmoid_of(F2 q) {
  return rcp2(add2(exp2_of<DT, false, -1>(q), both(1.f)));
}

// The parameters of a thread's column.
template <int DT>
struct Column {
  F2 gamma[4], beta[4];
  __device__ __forceinline__ void read(const GroupNormParams& P, int64_t ch, bool on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) gamma[i] = beta[i] = both(0.f);
    if (!on) return;
    Vec8<DT> v;
    load_pack(v, P.gamma + ch * ElemSize<DT>::value);
    unpack_pairs(v, gamma);
    if (P.norm == SP_NORM_LAYERNORM) {
      load_pack(v, P.beta + ch * ElemSize<DT>::value);
      unpack_pairs(v, beta);
    }
  }
};

// Sums over `width` neighbouring lanes (a power of two, aligned), N at once.
template <int N>
__device__ __forceinline__ void lanes_sum(float (&v)[N], int width) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    if (d >= width) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
  }
}
__device__ __forceinline__ float lanes_sum(float v, int width) {
  float w[1] = {v};
  lanes_sum(w, width);
  return w[0];
}

// n rows dealt to `parts` in turn: the k-th gets count(k), its first is first(k)
// when they are dealt in one piece each.  32-bit arithmetic: a 64-bit division
// costs a hundred instructions.
struct Deal {
  int each, extra;
  __device__ __forceinline__ Deal(int n, int parts) : each(n / parts), extra(n % parts) {}
  __device__ __forceinline__ int count(int k) const { return each + (k < extra ? 1 : 0); }
  __device__ __forceinline__ int first(int k) const { return k * each + (k < extra ? k : extra); }
};

// A vector that will be read once more before long: kept in L2 (load_pack's
// streaming loads give their lines up first).
template <int DT>
__device__ __forceinline__ void load_again(Vec8<DT>& p, const char* src) {
#pragma unroll
  for (int i = 0; i < Vec8<DT>::kBytes / 16; ++i) {
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(src) + i);
    p.w[4 * i] = v.x;
    p.w[4 * i + 1] = v.y;
    p.w[4 * i + 2] = v.z;
    p.w[4 * i + 3] = v.w;
  }
}

__device__ __forceinline__ float pair_sum(const F2 (&v)[4]) {
  const float2 w = split(add2(add2(v[0], v[1]), add2(v[2], v[3])));
  return w.x + w.y;
}

// The mean of values that sum to `sum`; inv: 1 / count rounded.  The product's error is
// taken off again, so that the mean of equal values is their value.  An infinity stays.
__device__ __forceinline__ float mean_of(float sum, float count, float inv) {
  const float m = sum * inv, near = fmaf(fmaf(-m, count, sum), inv, m);
  return isinf(m) ? m : near;
}

// x - m in place of a vector's x, before anything is multiplied: where all values are
// alike, however large, nothing is left (x rstd - m rstd would leave 2^-24 of m rstd).
__device__ __forceinline__ void centre(F2 (&x)[4], float m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = add2(x[i], both(-m));
}

// Sum of (x - m)^2 of a vector, which is left as x - m.
__device__ __forceinline__ float spread_sum(F2 (&x)[4], float m) {
  centre(x, m);
  F2 s = mul2(x[0], x[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fma2(x[i], x[i], s);
  const float2 w = split(s);
  return w.x + w.y;
}

__device__ __forceinline__ F2 neg(F2 v) { return mul2(v, both(-1.f)); }

// rstd folded into the column's gamma, for many vectors of one group (16-bit inputs).
template <int DT>
__device__ __forceinline__ void fold_rstd(Column<DT>& col, float rstd) {
  if constexpr (DT == SP_F32) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) col.gamma[i] = mul2(col.gamma[i], both(rstd));
}

// The result of one vector of x - mean; FOLDED: the column's gamma holds rstd.
template <int DT, bool FOLDED = false>
__device__ __forceinline__ Vec8<DT> norm_act(const F2 (&d)[4], float rstd, const Column<DT>& col,
                                             bool silu) {
  F2 y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const F2 z = FOLDED && DT != SP_F32 ? d[i] : mul2(d[i], both(rstd));
    y[i] = fma2(z, col.gamma[i], col.beta[i]);
  }
  if (silu) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], sigmoid_of<DT>(y[i]));
  }
  Vec8<DT> o;
  pack_pairs(o, y);
  return o;
}

// Running (count, mean, M2) of a thread's values.  A stretch of up to kStretch
// vectors sums x - k and its square for each of the 8 channels, k the
// stretch's first vector: one of the values themselves, so (x - k)^2 sums to at
// most the count times the spread, and no mean, however far from zero, costs
// digits.  Stretches then join by their means.  An infinity (which is no k) makes the
// mean infinite, as it would the sum.
constexpr int kStretch = 64;
struct Moments {
  F2 k[4], s[4], q[4];
  int n = 0;                          // vectors of the stretch
  float cnt = 0.f, mean = 0.f, m2 = 0.f;
  __device__ __forceinline__ void add(const F2 (&v)[4], bool centred) {
    if (n == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 w = split(v[i]);
        k[i] = centred ? f2(isinf(w.x) ? 0.f : -w.x, isinf(w.y) ? 0.f : -w.y) : both(0.f);
        s[i] = q[i] = both(0.f);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F2 d = add2(v[i], k[i]);
      s[i] = add2(s[i], d);
      q[i] = fma2(d, d, q[i]);
    }
    ++n;
  }
  // Ends the stretch.  Not centred: mean stays 0 and M2 is the sum of squares.
  __device__ __forceinline__ void join(bool centred) {
    if (n == 0) return;
    const float nf = static_cast<float>(n), inv = 1.f / nf;
    F2 mc[4], sum = both(0.f), rest = both(0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mc[i] = fma2(s[i], both(inv), neg(k[i]));              // the channel's mean
      sum = add2(sum, mc[i]);
      rest = add2(rest, centred ? fma2(neg(mul2(s[i], both(inv))), s[i], q[i]) : q[i]);
    }
    const float2 a = split(sum);
    const float mb = centred ? (a.x + a.y) * 0.125f : 0.f;
    F2 apart = both(0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F2 d = add2(mc[i], both(-mb));
      apart = fma2(d, d, apart);
    }
    const float2 r = split(rest), w = split(apart);
    const float nb = 8.f * nf, all = cnt + nb, part = nb / all, d = mb - mean;
    mean = isinf(d) ? mean + mb : fmaf(d, part, mean);
    m2 += (r.x + r.y) + (centred ? nf * (w.x + w.y) : 0.f) + d * d * cnt * part;
    cnt = all;
    n = 0;
  }
};

// Backward of one vector: z and dq (the gradient of q) in place of x and dy.
template <int DT>
__device__ __forceinline__ void back_act(F2 (&x)[4], F2 (&dy)[4], float mean, float rstd,
                                         const Column<DT>& col, bool silu) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = mul2(add2(x[i], both(-mean)), both(rstd));
  if (silu) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F2 q = fma2(x[i], col.gamma[i], col.beta[i]);
      const F2 s = sigmoid_of<DT>(q);
      const F2 t = fma2(mul2(s, both(-1.f)), s, s);          // s (1 - s)
      dy[i] = mul2(dy[i], fma2(q, t, s));                    // s + q s (1 - s)
    }
  }
}

// dx of one vector from its z and dq and the group's means of dz and dz z.
template <int DT>
__device__ __forceinline__ Vec8<DT> back_out(const F2 (&z)[4], const F2 (&dq)[4], float rstd,
                                             const Column<DT>& col, float m1, float m2) {
  F2 y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    y[i] = mul2(fma2(z[i], both(-m2), fma2(dq[i], col.gamma[i], both(-m1))), both(rstd));
  Vec8<DT> o;
  pack_pairs(o, y);
  return o;
}

// Adds the rows' parts of a column's parameter gradients (acc[0..3] dgamma,
// acc[4..7] dbeta) over the block in row order and writes the block's part.
// ch0, channels: the slab's first one and how many exist.
// buf: [rows][cols][17] floats of shared memory (17: the columns' banks differ).
__device__ __forceinline__ void put_param_part(const GroupNormParams& P, const F2 (&acc)[8],
                                               float* buf, int cx, int ry, int64_t ch0,
                                               int channels, int64_t part) {
  __syncthreads();
  if (ry < P.rows) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = split(acc[i]);
      buf[(ry * P.cols + cx) * 17 + 2 * i] = v.x;
      buf[(ry * P.cols + cx) * 17 + 2 * i + 1] = v.y;
    }
  }
  __syncthreads();
  const int64_t width = static_cast<int64_t>(P.t) * P.c;
  float* ws = P.ws + part * 2 * width + ch0;
  const int wide = P.cols * 8;
  for (int o = threadIdx.x; o < 2 * wide; o += blockDim.x) {
    const int beta = o >= wide ? 1 : 0, c = o - beta * wide;
    if (c >= channels) continue;
    const float* at = buf + (c >> 3) * 17 + beta * 8 + (c & 7);
    float v = 0.f;
#pragma unroll 8
    for (int k = 0; k < P.rows; ++k) v += at[k * P.cols * 17];
    ws[beta * width + c] = v;
  }
}

template <int MODE, int N>
struct RowSums {
  float values[MODE == kSumWarp ? kRowWarps : MODE == kSumTeam ? kRowMaxWarps : 1]
              [MODE == kSumWarp ? N : MODE == kSumTeam ? 2 * N : 1][MODE == kSumWarp ? 32 : 1];
};

// Sums v over the lanes (and warps) of the calling thread's group.
template <int MODE, int N>
struct RowGroup {
  RowSums<MODE, N>* sh;
  int q, warp, first_lane;            // first_lane: of the group (kSumWarp)
  int team_warps, team, parity = 0;   // kSumTeam
  __device__ __forceinline__ void sum(float (&v)[N]) {
    const int lane = threadIdx.x & 31;
    if constexpr (MODE == kSumLanes) {
      lanes_sum(v, q);
    } else if constexpr (MODE == kSumWarp) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        sh->values[warp][i][lane] = v[i];
        v[i] = 0.f;
      }
      __syncwarp();
      for (int j = 0; j < q; ++j) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += sh->values[warp][i][first_lane + j];
      }
    } else {
      lanes_sum(v, 32);
      const int at = parity * N;      // two buffers: the next sum may begin at once
      parity ^= 1;
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) sh->values[warp][at + i][0] = v[i];
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(team_warps * 32) : "memory");
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = 0.f;
      for (int w = 0; w < team_warps; ++w) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += sh->values[team * team_warps + w][at + i][0];
      }
    }
  }
};

// Calls use(index) for a lane's share of the rows x q entries of group g in
// [rows][cols] shared memory: a lane a row where there are many rows, else the
// lanes along the group.
template <typename Use>
__device__ __forceinline__ void group_entries(const GroupNormParams& P, int g, Use use) {
  const int lane = threadIdx.x & 31;
  if (P.rows >= 16) {
    for (int y = lane; y < P.rows; y += 32)
      for (int j = 0; j < P.q; ++j) use(y, y * P.cols + g * P.q + j);
  } else {
    for (int y = 0; y < P.rows; ++y)
      for (int j = lane; j < P.q; j += 32) use(y, y * P.cols + g * P.q + j);
  }
}

// The two halves of a cluster barrier: between them a block may not touch a
// partner's shared memory, but goes on with its own work.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

}  // namespace spb
