// Gated recurrence, backward.  With q the gradient reaching a token's state
// from the token after it (at the end of a sequence the gradient of its last
// state), from the last token to the first
//   dh[i] = dy[i] + q,   q' = a[i] dh[i]   (at a sequence's first token q' = dh0)
//   dgate[i] = dh[i] a[i] k[i] (h[i-1] - v[i])  (tied)   or  dh[i] a[i] k[i] h[i-1]
//   dvalue[i] = dh[i] k[i]                      (tied)   or  dh[i]
// The states h are computed again from the forward's state at the start of
// each run, in float32: that reads a quarter byte an element instead of the
// two of the rounded output, and the difference h - v keeps its digits.
#include "scan.cuh"

namespace spb {

template <int DT, bool TIED, bool PACKED>
__global__ void __launch_bounds__(32 * kScanMaxWarps) scan_bwd_kernel(const ScanParams P) {
  constexpr int E = ElemSize<DT>::value;
  extern __shared__ float2 slots[];                  // [warps][16][32]
  __shared__ ScanShared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int C = P.cluster, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  if (C > 1) cluster_sync_all();                     // the partners run: their shared memory is there
  pdl_wait();
  int unit = static_cast<int>(blockIdx.x) / C;
  if (PACKED && blockIdx.x == 0 && warp == 0)
    check_cu_seqlens(P.cu_seqlens, P.n_seqs, P.s, P.status);
  const int slab = unit % P.slabs;
  unit /= P.slabs;
  const int r = unit % P.t, bi = unit / P.t;
  const int ch = slab * kScanChannels + 2 * lane;
  const bool on = ch < P.c;
  const int64_t col = static_cast<int64_t>(ch) * E;
  const char* gate = P.gate[r] + bi * P.s * P.ld_gate + col;
  const char* value = P.value[r] + bi * P.s * P.ld_value + col;
  const char* dy = P.dy[r] + bi * P.s * P.ld_dy + col;
  char* dgate = P.out[r] + bi * P.s * P.ld_out + col;
  char* dvalue = P.dvalue[r] + bi * P.s * P.ld_dvalue + col;
  const int64_t n_runs = (P.s + kScanRun - 1) / kScanRun;
  const float* states = P.states[r] + bi * n_runs * P.c + ch;
  float2(*slot)[32] = reinterpret_cast<float2(*)[32]>(slots + warp * kScanRun * 32);
  if (PACKED && rank == 0) pass_empty(P, P.dhT[r], P.hT[r], ch, on);

  const int64_t stretch = static_cast<int64_t>(C) * nw * kScanRun;
  const int64_t last = (P.s - 1) / stretch * stretch;
  float2 carry = make_float2(0.f, 0.f);
  int par = 0;
  for (int64_t base = last; base >= 0; base -= stretch, par ^= 1) {
    const int64_t tok0 = base + static_cast<int64_t>(rank * nw + warp) * kScanRun;
    Two<DT> draw[kScanRun];
    float k[kScanRun][2], dg[kScanRun][2];           // k, and dgate without its factor dh
    const RunMarks marks = run_marks<PACKED>(P, tok0);
    fetch_states<PACKED>(P, P.h0[r], marks.starts, tok0, bi, ch, on, slot);
    {
      Two<DT> graw[kScanRun], vraw[kScanRun];
      float2 st = make_float2(0.f, 0.f);
      // tokens after the last one take part as zeros
#pragma unroll
      for (int i = 0; i < kScanRun; ++i) {
        graw[i] = vraw[i] = draw[i] = Two<DT>{};
        if (on && tok0 + i < P.s) {
          load_pack(graw[i], gate + (tok0 + i) * P.ld_gate);
          load_pack(vraw[i], value + (tok0 + i) * P.ld_value);
          load_pack(draw[i], dy + (tok0 + i) * P.ld_dy);
        }
      }
      if (on && tok0 < P.s)
        st = __ldcs(reinterpret_cast<const float2*>(states + (tok0 / kScanRun) * P.c));
      float h[2] = {st.x, st.y};
#pragma unroll
      for (int i = 0; i < kScanRun; ++i) {
        if ((marks.starts >> i) & 1u) {
          const float2 v = slot[i][lane];
          h[0] = v.x;
          h[1] = v.y;
        }
        float g[2], v[2];
        unpack(graw[i], g);
        unpack(vraw[i], v);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float a;
          gate_of<DT>(g[e], a, k[i][e]);
          const float d = TIED ? v[e] - h[e] : h[e];
          dg[i][e] = a * k[i][e] * (TIED ? -d : d);
          h[e] = TIED ? fmaf(k[i][e], d, h[e]) : fmaf(a, d, v[e]);
        }
      }
    }
    fetch_states<PACKED>(P, P.dhT[r], marks.ends, tok0, bi, ch, on, slot);
    // q leaving the run's first token as a map of the q entering its last one
    float q[2] = {0.f, 0.f}, fac[2] = {1.f, 1.f};
#pragma unroll
    for (int i = kScanRun - 1; i >= 0; --i) {
      if ((marks.ends >> i) & 1u) {
        const float2 v = slot[i][lane];
        q[0] = v.x;
        q[1] = v.y;
        fac[0] = fac[1] = 0.f;
      }
      float d[2];
      unpack(draw[i], d);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = d[e] + q[e];
        q[e] = fmaf(-k[i][e], x, x);                 // a x
        fac[e] = fmaf(-k[i][e], fac[e], fac[e]);
      }
    }
    const Map2 mine{fac[0], fac[1], q[0], q[1]};
    float2 in = join_runs<PACKED, -1>(sh, par, mine, C, rank, carry);
    if (tok0 >= P.s) continue;
#pragma unroll
    for (int i = kScanRun - 1; i >= 0; --i) {
      if ((marks.ends >> i) & 1u) in = slot[i][lane];
      float d[2], o[2];
      unpack(draw[i], d);
      d[0] += in.x;
      d[1] += in.y;
      in.x = fmaf(-k[i][0], d[0], d[0]);
      in.y = fmaf(-k[i][1], d[1], d[1]);
      if ((marks.starts >> i) & 1u) slot[i][lane] = make_float2(d[0], d[1]);
      if (on && tok0 + i < P.s) {
        Two<DT> w;
        o[0] = d[0] * dg[i][0];
        o[1] = d[1] * dg[i][1];
        pack(w, o);
        store_pack(dgate + (tok0 + i) * P.ld_out, w);
        o[0] = TIED ? d[0] * k[i][0] : d[0];
        o[1] = TIED ? d[1] * k[i][1] : d[1];
        pack(w, o);
        store_pack(dvalue + (tok0 + i) * P.ld_dvalue, w);
      }
    }
    if (P.hT[r] != nullptr && marks.starts != 0) {
      // dh0 = a dh: a from the gate again, where 1 - k would lose a small one
      uint32_t left = marks.starts;
      while (left != 0) {
        const int i = __ffs(left) - 1;
        left &= left - 1;
        if (!on) continue;
        Two<DT> graw;
        load_pack(graw, gate + (tok0 + i) * P.ld_gate);
        float g[2], a[2], kk;
        unpack(graw, g);
        gate_of<DT>(g[0], a[0], kk);
        gate_of<DT>(g[1], a[1], kk);
        const float2 d = slot[i][lane];
        slot[i][lane] = make_float2(a[0] * d.x, a[1] * d.y);
      }
      put_states<PACKED>(P, P.hT[r], marks.starts, tok0, bi, ch, on, slot);
    }
  }
}

template <int DT>
static const void* scan_bwd_fn(bool tied, bool packed) {
  if (tied)
    return packed ? reinterpret_cast<const void*>(&scan_bwd_kernel<DT, true, true>)
                  : reinterpret_cast<const void*>(&scan_bwd_kernel<DT, true, false>);
  return packed ? reinterpret_cast<const void*>(&scan_bwd_kernel<DT, false, true>)
                : reinterpret_cast<const void*>(&scan_bwd_kernel<DT, false, false>);
}

cudaError_t launch_scan_bwd(ScanParams p, int dtype, cudaStream_t st) {
  void* args[] = {&p};
  const bool packed = p.cu_seqlens != nullptr;
  int warps;
  scan_shape(p, &warps, &p.cluster);
  const void* fn = dtype == SP_BF16  ? scan_bwd_fn<SP_BF16>(p.tied, packed)
                   : dtype == SP_F16 ? scan_bwd_fn<SP_F16>(p.tied, packed)
                                     : scan_bwd_fn<SP_F32>(p.tied, packed);
  return launch_scan(fn, p, warps, args, st);
}

}  // namespace spb
