// Shared parts of group norm with an activation, channels last:
//   z = (x - mean) rstd over the l rows and c / groups channels of a group of
//   one sample,  q = z gamma + beta,  y = q or q sigmoid(q).
//
// A thread owns one vector of 8 channels (its column; all of one group) and
// walks rows, so the parameters and their gradients stay in registers.  Two
// forms, by the size of a sample:
//  - tiles: a block takes whole samples of few rows; every thread holds its
//    vectors in registers between the statistics and the result;
//  - units: a cluster of blocks takes one sample's slab of groups, keeps the
//    rows it can in shared memory and reads the rest again (from L2 where the
//    cluster's share fits it), and joins its statistics through distributed
//    shared memory.
// Sums run in a fixed order: results do not depend on timing.  Statistics are
// two-pass (of values held in registers) and joined as (count, mean, M2), so a
// mean far above the spread costs no digits.
#pragma once

#include "region.cuh"

namespace spb {

template <int DT>
using Vec8 = Pack<DT, 8>;

template <int DT>
__device__ __forceinline__ float sigmoid_of(float q) {
  if constexpr (DT == SP_F32) {
    return __frcp_rn(1.f + expf(-q));
  } else {
    // 16-bit results: the fast exponential's error is far below their rounding
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(q * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
    return s;
  }
}

// The parameters of a thread's column.
template <int DT>
struct Column {
  float gamma[8], beta[8];
  __device__ __forceinline__ void read(const GroupNormParams& P, int64_t ch, bool on) {
#pragma unroll
    for (int i = 0; i < 8; ++i) gamma[i] = beta[i] = 0.f;
    if (!on) return;
    Vec8<DT> v;
    load_pack(v, P.gamma + ch * ElemSize<DT>::value);
    unpack(v, gamma);
    if (P.norm == SP_NORM_LAYERNORM) {
      load_pack(v, P.beta + ch * ElemSize<DT>::value);
      unpack(v, beta);
    }
  }
};

// Sum over `width` neighbouring lanes (a power of two, aligned).
__device__ __forceinline__ float lanes_sum(float v, int width) {
  for (int d = width >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

template <int DT>
__device__ __forceinline__ void norm_act(const float (&x)[8], float mean, float rstd,
                                         const Column<DT>& col, bool silu, Vec8<DT>& o) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = fmaf((x[i] - mean) * rstd, col.gamma[i], col.beta[i]);
    y[i] = silu ? q * sigmoid_of<DT>(q) : q;
  }
  pack(o, y);
}

// Backward of one vector: z and dq gamma (the gradient of z) from x and dy,
// adding the vector's part of the parameter gradients.
template <int DT>
__device__ __forceinline__ void back_act(const float (&x)[8], const float (&dy)[8], float mean,
                                         float rstd, const Column<DT>& col, bool silu,
                                         float (&z)[8], float (&dq)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    z[i] = (x[i] - mean) * rstd;
    dq[i] = dy[i];
    if (silu) {
      const float q = fmaf(z[i], col.gamma[i], col.beta[i]);
      const float s = sigmoid_of<DT>(q);
      dq[i] *= s * fmaf(q, 1.f - s, 1.f);
    }
  }
}

// Adds the rows' parts of a column's parameter gradients (acc[0..7] dgamma,
// acc[8..15] dbeta) over the block in row order and writes the block's part.
// buf: [rows][cols][17] floats of shared memory (17: the columns' banks differ).
__device__ __forceinline__ void put_param_part(const GroupNormParams& P, const float (&acc)[16],
                                               float* buf, int cx, int ry, bool on, int64_t ch,
                                               int64_t part) {
  __syncthreads();
  if (ry < P.rows) {
#pragma unroll
    for (int i = 0; i < 16; ++i) buf[(ry * P.cols + cx) * 17 + i] = acc[i];
  }
  __syncthreads();
  if (ry != 0 || !on) return;
  const int64_t width = static_cast<int64_t>(P.t) * P.c;
  float* ws = P.ws + part * 2 * width + ch;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float v = 0.f;
    for (int k = 0; k < P.rows; ++k) v += buf[(k * P.cols + cx) * 17 + i];
    ws[(i / 8) * width + (i & 7)] = v;
  }
}

}  // namespace spb
