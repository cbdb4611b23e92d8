// Device helpers of the operators between g and the next g* (rotary
// positions, gated recurrence, group norm): element types and packed loads.
//
// These tensors hold the whole sequence and one rank's channels.  DT is an
// sp_dtype_t: bf16, fp16 or float32 elements; all arithmetic is float32, each
// stored value rounded once.
#pragma once

#include <cuda_fp16.h>

#include "host_common.h"
#include "region.h"
#include "sp_device.cuh"

namespace spb {

template <int DT>
struct ElemSize {
  static constexpr int value = DT == SP_F32 ? 4 : 2;
};

// N consecutive elements as 32-bit words (N * size >= 4) or one 16-bit value.
template <int DT, int N>
struct Pack {
  static constexpr int kBytes = N * ElemSize<DT>::value;
  static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
  uint32_t w[kWords];
};

// Read-once / write-once accesses of a pack in pieces of at most 16 bytes
// (plain coherent loads: an output may be the input itself where an entry
// point allows it).
template <int DT, int N>
__device__ __forceinline__ void load_pack(Pack<DT, N>& p, const char* src) {
  constexpr int B = Pack<DT, N>::kBytes;
  if constexpr (B >= 16) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src) + i);
      p.w[4 * i] = v.x;
      p.w[4 * i + 1] = v.y;
      p.w[4 * i + 2] = v.z;
      p.w[4 * i + 3] = v.w;
    }
  } else if constexpr (B == 8) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(src));
    p.w[0] = v.x;
    p.w[1] = v.y;
  } else if constexpr (B == 4) {
    p.w[0] = __ldcs(reinterpret_cast<const unsigned int*>(src));
  } else {
    p.w[0] = __ldcs(reinterpret_cast<const unsigned short*>(src));
  }
}

template <int DT, int N>
__device__ __forceinline__ void store_pack(char* dst, const Pack<DT, N>& p) {
  constexpr int B = Pack<DT, N>::kBytes;
  if constexpr (B >= 16) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i)
      __stcs(reinterpret_cast<uint4*>(dst) + i,
             make_uint4(p.w[4 * i], p.w[4 * i + 1], p.w[4 * i + 2], p.w[4 * i + 3]));
  } else if constexpr (B == 8) {
    __stcs(reinterpret_cast<uint2*>(dst), make_uint2(p.w[0], p.w[1]));
  } else if constexpr (B == 4) {
    __stcs(reinterpret_cast<unsigned int*>(dst), p.w[0]);
  } else {
    __stcs(reinterpret_cast<unsigned short*>(dst), static_cast<unsigned short>(p.w[0]));
  }
}

__device__ __forceinline__ float half_bits(uint32_t v) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(v)));
}

template <int DT, int N>
__device__ __forceinline__ void unpack(const Pack<DT, N>& p, float (&f)[N]) {
  if constexpr (DT == SP_F32) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __uint_as_float(p.w[i]);
  } else if constexpr (DT == SP_BF16) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      f[i] = __uint_as_float((i & 1) ? (p.w[i / 2] & 0xFFFF0000u) : (p.w[i / 2] << 16));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = half_bits((i & 1) ? (p.w[i / 2] >> 16) : p.w[i / 2]);
  }
}

template <int DT>
__device__ __forceinline__ uint32_t pair_bits(float lo, float hi) {
  uint32_t r;
  if constexpr (DT == SP_BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int DT, int N>
__device__ __forceinline__ void pack(Pack<DT, N>& p, const float (&f)[N]) {
  if constexpr (DT == SP_F32) {
#pragma unroll
    for (int i = 0; i < N; ++i) p.w[i] = __float_as_uint(f[i]);
  } else if constexpr (N == 1) {
    p.w[0] = pair_bits<DT>(f[0], 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) p.w[i] = pair_bits<DT>(f[2 * i], f[2 * i + 1]);
  }
}

// Packed pairs of floats: one instruction for both.
using F2 = unsigned long long;

__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(F2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// N elements as N / 2 pairs, and back (each rounded once).
template <int DT, int N>
__device__ __forceinline__ void unpack_pairs(const Pack<DT, N>& p, F2 (&v)[N / 2]) {
  float f[N];
  unpack(p, f);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) v[i] = f2(f[2 * i], f[2 * i + 1]);
}
template <int DT, int N>
__device__ __forceinline__ void pack_pairs(Pack<DT, N>& p, const F2 (&v)[N / 2]) {
  float f[N];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float2 w = split(v[i]);
    f[2 * i] = w.x;
    f[2 * i + 1] = w.y;
  }
  pack(p, f);
}

// The packed sequence of token `tok`: the largest j < n with cu[j] <= tok (the
// last of several sequences that begin there: the others are empty).  One
// warp, 32 probes a step; in bounds whatever cu holds.
__device__ __forceinline__ int seq_of_token(const int32_t* cu, int n, int64_t tok) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int at = lo + lane * step;
    const bool le = at < lo + len && static_cast<int64_t>(__ldg(cu + at)) <= tok;
    const int cnt = __popc(__ballot_sync(0xFFFFFFFFu, le));
    const int skip = cnt > 0 ? (cnt - 1) * step : 0;
    lo += skip;
    len = len - skip < step ? len - skip : step;
  }
  return lo;
}

// 1 / v of both, within an ulp; subnormal results are flushed.
__device__ __forceinline__ F2 rcp2(F2 v) {
  float2 x = split(v);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x.y));
  return f2(x.x, x.y);
}

// exp of both, for results of type DT: 2^t with t = g log2(e) rounded.  The
// rounding's part, 2^-24 of t, is far below 16-bit results' own; for float32 ones
// 2^t is multiplied by 1 + r ln 2, where r = g log2(e) - t comes from the constant
// split in two parts (as in Cody and Waite's argument reductions), and the power's own
// error of 2^-22 stays, beside the 2^-23 of a sigmoid's reciprocal: float32 SiLU is off
// by at most 4.3 2^-24 between -80 and 80, torch's by 2.4.  (The library's exponential
// and reciprocal took half as long again for the whole recurrence: 4 x 65,536 tokens of
// 256 float32 channels 244 us, so 168.)  Float32 arguments are held where the products
// are finite: 1 / (1 + exp(88.7)) is flushed to zero already, and exp(-104) too.  CAP
// (float32): exp(87) at most, whose reciprocal is still normal.
// SIGN: of exp(SIGN g); the bounds are those of SIGN g.
template <int DT, bool CAP, int SIGN = 1>
__device__ __forceinline__ F2 exp2_of(F2 g) {
  const F2 log2e = f2(SIGN * 1.4426950408889634f, SIGN * 1.4426950408889634f);
  float2 x;
  F2 rest = f2(0.f, 0.f);
  if constexpr (DT == SP_F32) {
    if constexpr (SIGN < 0) g = mul2(g, f2(-1.f, -1.f));
    x = split(g);
    asm("max.NaN.f32 %0, %0, 0fC2D00000;" : "+f"(x.x));     // -104
    asm("max.NaN.f32 %0, %0, 0fC2D00000;" : "+f"(x.y));
    if constexpr (CAP) {
      asm("min.NaN.f32 %0, %0, 0f42AE0000;" : "+f"(x.x));   // 87
      asm("min.NaN.f32 %0, %0, 0f42AE0000;" : "+f"(x.y));
    } else {
      asm("min.NaN.f32 %0, %0, 0f42B16666;" : "+f"(x.x));   // 88.7
      asm("min.NaN.f32 %0, %0, 0f42B16666;" : "+f"(x.y));
    }
    g = f2(x.x, x.y);
    const F2 t = mul2(g, f2(1.4426950408889634f, 1.4426950408889634f));
    rest = fma2(g, f2(-1.4426950408889634f, -1.4426950408889634f), t);
    rest = fma2(g, f2(-1.92596299e-8f, -1.92596299e-8f), rest);
    rest = mul2(rest, f2(-0.69314718f, -0.69314718f));
    x = split(t);
  } else {
    static_assert(!CAP, "16-bit arguments are held by their users");
    x = split(mul2(g, log2e));
  }
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x.y));
  const F2 e = f2(x.x, x.y);
  if constexpr (DT == SP_F32) return fma2(e, rest, e);
  return e;
}

}  // namespace spb
