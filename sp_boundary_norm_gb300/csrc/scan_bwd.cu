// Gated recurrence, backward.  With q the gradient reaching a token's state
// from the token after it (at the end of a sequence the gradient of its last
// state), from the last token to the first
//   dh[i] = dy[i] + q,   q' = a[i] dh[i]   (at a sequence's first token q' = dh0)
//   dgate[i] = dh[i] a[i] k[i] (h[i-1] - v[i])  (tied)   or  dh[i] a[i] k[i] h[i-1]
//   dvalue[i] = dh[i] k[i]                      (tied)   or  dh[i]
// The states h are computed again from the forward's state at the start of
// each run, in float32: that reads a quarter byte an element instead of the
// two of the rounded output, and the difference h - v keeps its digits.  Bound by
// HBM for many channels, 84 % of the measured copy rate (scan.cuh has the
// figures); three blocks an SM, because a run's 40 factors stay in registers
// between the two directions.
#include "scan.cuh"

namespace spb {

// Blocks an SM that the registers are held to (8 ranks of 8 rows of 2048 tokens x 1024
// channels: three 235 us, two 256, four, with spilled registers, 317).
constexpr int kBwdBlocks = 3;

// The run's factors, from its rows in shared memory: e = exp(-gate), from which the
// way back takes a and k again (both kept would cost 32 registers more), and
// dg = a k (h[i-1] - v[i]) or a k h[i-1], dgate without its factor dh.  i0, h0: the
// first token that begins a sequence and the state before it; begin(i): that before any
// other.  Returns q leaving the run's first token as a map of the q entering its last
// one, gathered on the way: with A[i] the product of a[0 .. i],
//   q leaving = sum over i of A[i] dy[i] + A[15] q entering,
// up to the first token i1 that ends a sequence, which q1 enters.
template <int DT, bool TIED, int KIND, typename Shared, typename Begin>
__device__ __forceinline__ Map2 back_factors(const Shared& sh, int stage, uint32_t starts,
                                             int i0, F2 h0, int i1, F2 q1, F2 h,
                                             F2 (&e)[kScanRun], F2 (&dg)[kScanRun],
                                             Two<DT> (&dy)[kScanRun], Begin begin) {
  F2 q = f2(0.f, 0.f);
  RunFactor fac;
#pragma unroll
  for (int i = 0; i < kScanRun; ++i) {
    if (KIND == kSingleRun && i == i0) h = h0;
    if (KIND == kAnyRun && ((starts >> i) & 1u)) h = i == i0 ? h0 : begin(i);
    const F2 a = open_gate<DT>(sh.template raw<DT>(stage, 0, i), e[i]), k = mul2(e[i], a);
    const F2 v = sh.template row<DT>(stage, 1, i);
    // a k first: k k, or d times either, may underflow where the product does not
    dg[i] = mul2(mul2(k, a), TIED ? fma2(v, f2(-1.f, -1.f), h) : h);
    h = next_state<TIED>(a, k, h, v);
    dy[i] = sh.template raw<DT>(stage, 2, i);
    // (i1 = -1: no end)
    if (KIND == kPlainRun || static_cast<uint32_t>(i) <= static_cast<uint32_t>(i1)) {
      fac.next(a, k);
      q = fma2(fac.a, unpack2<DT>(dy[i]), q);
      if (KIND != kPlainRun && i == i1) q = fma2(fac.a, q1, q);
    }
  }
  if (KIND != kPlainRun && i1 >= 0) fac.cut();
  return Map2{fac.whole(), q};
}

template <int DT, bool TIED, bool PACKED, bool WIDE>
__global__ void __launch_bounds__(32 * (WIDE ? kScanWideWarps : kScanWarps), WIDE ? 1 : kBwdBlocks)
scan_bwd_kernel(const ScanParams P) {
  constexpr int E = ElemSize<DT>::value;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
  const int nw = blockDim.x >> 5;
  const int C = P.cluster, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const ScanShared<E, 3> sh(smem, warp, nw, C);
  if (C > 1) cluster_sync_all(); else __syncthreads();   // mbarriers (and partners) are ready
  pdl_wait();
  int unit = static_cast<int>(blockIdx.x) / C;
  if (PACKED && blockIdx.x == 0 && warp == 0)
    check_cu_seqlens(P.cu_seqlens, P.n_seqs, P.s, P.status);
  const int slab = unit % P.slabs;
  unit /= P.slabs;
  const int r = unit % P.t, bi = unit / P.t;
  const int ch0 = slab * kScanChannels, ch = ch0 + 2 * lane;
  const bool on = ch < P.c;
  const int bytes = (P.c - ch0 < kScanChannels ? P.c - ch0 : kScanChannels) * E;
  const int64_t row0 = bi * P.s, col0 = static_cast<int64_t>(ch0) * E;
  const int64_t col = static_cast<int64_t>(ch) * E;
  const char* gate = P.gate[r] + row0 * P.ld_gate + col0;
  const char* value = P.value[r] + row0 * P.ld_value + col0;
  const char* dy_at = P.dy[r] + row0 * P.ld_dy + col0;
  char* dgate = P.out[r] + row0 * P.ld_out + col;
  char* dvalue = P.dvalue[r] + row0 * P.ld_dvalue + col;
  const int64_t n_runs = (P.s + kScanRun - 1) / kScanRun;
  const float* states = P.states[r] + bi * n_runs * P.c + ch;
  if (PACKED && rank == 0) pass_empty(P, P.dhT[r], P.hT[r], ch, on);

  const int64_t stretch = static_cast<int64_t>(C) * nw * kScanRun;
  const int64_t last = (P.s - 1) / stretch * stretch;
  int64_t tok0 = last + static_cast<int64_t>(rank * nw + warp) * kScanRun;
  // tokens after the last one take part as zeros
  auto fetch = [&](int stage, int64_t at) {
    sh.copy(stage, 0, gate, P.ld_gate, at, P.s, bytes);
    sh.copy(stage, 1, value, P.ld_value, at, P.s, bytes);
    sh.copy(stage, 2, dy_at, P.ld_dy, at, P.s, bytes);
    cp_async_commit();
  };
  float2 entering = make_float2(0.f, 0.f);           // the state entering the next run
  auto fetch_entering = [&](int64_t at) {
    if (on && at >= 0 && at < P.s)
      entering = __ldcs(reinterpret_cast<const float2*>(states + (at / kScanRun) * P.c));
  };
#pragma unroll
  for (int k = 0; k < kStages; ++k) fetch(k, tok0 - k * stretch);
  fetch_entering(tok0);
  F2 carry = f2(0.f, 0.f);
  SeqWindow win = no_window();
  int step = 0;
  int late = kNever;
  for (int64_t base = last; base >= 0; base -= stretch, tok0 -= stretch, ++step) {
    const RunMarks marks = run_marks<PACKED>(P, tok0, win, sh.first, 15);
    const int kind = run_kind(marks, P.s - tok0);
    auto seq = [&](int i) { return seq_of_run<PACKED>(win, sh.first, marks.starts, bi, i); };
    auto begin = [&](int i) { return load_state(P.h0[r], seq(i), P.c, ch, on); };
    auto end = [&](int i) { return load_state(P.dhT[r], seq(i), P.c, ch, on); };
    // (the first beginning's state and the first end's gradient are asked for
    // beneath the wait for the rows)
    const int i0 = __ffs(marks.starts) - 1, i1 = __ffs(marks.ends) - 1;
    F2 h0 = f2(0.f, 0.f), q1 = h0;
    if (i0 >= 0) h0 = begin(i0);
    if (i1 >= 0) q1 = end(i1);
    Two<DT> dy[kScanRun];
    F2 e[kScanRun], dg[kScanRun];
    sh.wait();
    const int stage = step % kStages;
    const F2 h = f2(entering.x, entering.y);
    Map2 mine;
    if (kind == kPlainRun)
      mine = back_factors<DT, TIED, kPlainRun>(sh, stage, 0u, 0, h0, 0, q1, h, e, dg, dy, begin);
    else if (kind == kSingleRun)
      mine = back_factors<DT, TIED, kSingleRun>(sh, stage, 0u, i0, h0, i1, q1, h, e, dg, dy, begin);
    else
      mine = back_factors<DT, TIED, kAnyRun>(sh, stage, marks.starts, i0, h0, i1, q1, h, e, dg, dy,
                                             begin);
    __syncwarp();                     // every lane has read the rows
    fetch(stage, tok0 - kStages * stretch);
    fetch_entering(tok0 - stretch);
    F2 into = join_runs<PACKED, -1>(sh.join, step, mine, marks.ends != 0u, C, rank, warp, nw,
                                    P.withhold, carry, late);
    if (tok0 >= P.s) continue;
    char* at_g = dgate + tok0 * P.ld_out;
    char* at_v = dvalue + tok0 * P.ld_dvalue;
    // token i's gradients from the q entering it; leaves the q before it
    auto back = [&](int i, bool there) {
      const F2 a = rcp2(add2(e[i], f2(1.f, 1.f)));
      const F2 dh = add2(unpack2<DT>(dy[i]), into);
      into = mul2(a, dh);
      if (!there) return;
      store_pack(at_g + static_cast<uint64_t>(P.ld_out) * i, pack2<DT>(mul2(dh, dg[i])));
      store_pack(at_v + static_cast<uint64_t>(P.ld_dvalue) * i,
                 pack2<DT>(TIED ? mul2(mul2(e[i], a), dh) : dh));
    };
    if (kind == kPlainRun) {
      if (on) {
#pragma unroll
        for (int i = kScanRun - 1; i >= 0; --i) back(i, true);
      }
    } else if (kind == kSingleRun) {
      F2 first = f2(0.f, 0.f);
#pragma unroll
      for (int i = kScanRun - 1; i >= 0; --i) {
        if (i == i1) into = q1;
        back(i, on);
        if (i == i0) first = into;
      }
      if (i0 >= 0) store_state(P.hT[r], seq(i0), P.c, ch, on, first);
    } else {
      const int rows = P.s - tok0 < kScanRun ? static_cast<int>(P.s - tok0) : kScanRun;
#pragma unroll
      for (int i = kScanRun - 1; i >= 0; --i) {
        if ((marks.ends >> i) & 1u) into = i == i1 ? q1 : end(i);
        back(i, on && i < rows);
        if ((marks.starts >> i) & 1u) store_state(P.hT[r], seq(i), P.c, ch, on, into);
      }
    }
  }
  cp_async_wait<0>();
  if (C > 1) leave_cluster<-1>(sh.join, C, warp, nw, late, step, P.status);
}

template <int DT, bool WIDE>
static const void* scan_bwd_fn(bool tied, bool packed) {
  if (tied)
    return packed ? reinterpret_cast<const void*>(&scan_bwd_kernel<DT, true, true, WIDE>)
                  : reinterpret_cast<const void*>(&scan_bwd_kernel<DT, true, false, WIDE>);
  return packed ? reinterpret_cast<const void*>(&scan_bwd_kernel<DT, false, true, WIDE>)
                : reinterpret_cast<const void*>(&scan_bwd_kernel<DT, false, false, WIDE>);
}

template <bool WIDE>
static const void* scan_bwd_fn(int dtype, bool tied, bool packed) {
  return dtype == SP_BF16  ? scan_bwd_fn<SP_BF16, WIDE>(tied, packed)
         : dtype == SP_F16 ? scan_bwd_fn<SP_F16, WIDE>(tied, packed)
                           : scan_bwd_fn<SP_F32, WIDE>(tied, packed);
}

cudaError_t launch_scan_bwd(ScanParams p, int dtype, cudaStream_t st) {
  void* args[] = {&p};
  const bool packed = p.cu_seqlens != nullptr;
  const ScanKernels kernels{scan_bwd_fn<false>(dtype, p.tied, packed), nullptr,
                            scan_bwd_fn<true>(dtype, p.tied, packed)};
  const ScanCost cost = dtype == SP_F32 ? ScanCost{0.95, 1.34, 0.08, 0.3, 3, 5}
                                        : ScanCost{0.46, 0.81, 0.06, 0.18, 3, 5};
  return launch_scan(kernels, p, dtype == SP_F32 ? 4 : 2, cost, args, st);
}

}  // namespace spb
