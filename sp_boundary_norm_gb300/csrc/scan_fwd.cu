// Gated recurrence, forward: y, the last state of every sequence, and the
// state entering every run of 16 tokens for the backward.  One token of every
// sequence (a decoding step) takes a kernel without the joins.
#include "scan.cuh"

namespace spb {

template <int DT, bool TIED, bool PACKED>
__global__ void __launch_bounds__(32 * kScanMaxWarps) scan_fwd_kernel(const ScanParams P) {
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
  const char* gate = P.gate[r] + bi * P.s * P.ld_gate + static_cast<int64_t>(ch) * E;
  const char* value = P.value[r] + bi * P.s * P.ld_value + static_cast<int64_t>(ch) * E;
  char* out = P.out[r] + bi * P.s * P.ld_out + static_cast<int64_t>(ch) * E;
  const int64_t n_runs = (P.s + kScanRun - 1) / kScanRun;
  float* states = P.states[r];
  if (states != nullptr) states += bi * n_runs * P.c + ch;
  float2(*slot)[32] = reinterpret_cast<float2(*)[32]>(slots + warp * kScanRun * 32);
  if (PACKED && rank == 0) pass_empty(P, P.h0[r], P.hT[r], ch, on);

  Two<DT> graw[kScanRun], vraw[kScanRun];
  const int64_t stretch = static_cast<int64_t>(C) * nw * kScanRun;
  int64_t tok0 = static_cast<int64_t>(rank * nw + warp) * kScanRun;
  auto fetch = [&](int64_t at) {
#pragma unroll
    for (int i = 0; i < kScanRun; ++i) {
      if (on && at + i < P.s) {
        load_pack(graw[i], gate + (at + i) * P.ld_gate);
        load_pack(vraw[i], value + (at + i) * P.ld_value);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kScanRun; ++i) graw[i] = vraw[i] = Two<DT>{};
  fetch(tok0);
  float2 carry = make_float2(0.f, 0.f);
  int par = 0;
  for (int64_t base = 0; base < P.s; base += stretch, tok0 += stretch, par ^= 1) {
    const RunMarks marks = run_marks<PACKED>(P, tok0);
    fetch_states<PACKED>(P, P.h0[r], marks.starts, tok0, bi, ch, on, slot);
    float h[kScanRun][2], f[kScanRun][2];            // h = h[i] + f[i] * (state entering)
    float cur[2] = {0.f, 0.f}, fac[2] = {1.f, 1.f};
#pragma unroll
    for (int i = 0; i < kScanRun; ++i) {
      if ((marks.starts >> i) & 1u) {
        const float2 v = slot[i][lane];
        cur[0] = v.x;
        cur[1] = v.y;
        fac[0] = fac[1] = 0.f;
      }
      float g[2], v[2];
      unpack(graw[i], g);
      unpack(vraw[i], v);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float a, k;
        gate_of<DT>(g[e], a, k);
        cur[e] = TIED ? fmaf(k, v[e] - cur[e], cur[e]) : fmaf(a, cur[e], v[e]);
        fac[e] = fac[e] * a;
        h[i][e] = cur[e];
        f[i][e] = fac[e];
      }
    }
    fetch(tok0 + stretch);
    const Map2 mine{fac[0], fac[1], cur[0], cur[1]};
    const float2 in = join_runs<PACKED, 1>(sh, par, mine, C, rank, carry);
    if (tok0 >= P.s) continue;
    if (states != nullptr && on)
      __stcs(reinterpret_cast<float2*>(states + (tok0 / kScanRun) * P.c), in);
    const uint32_t ends = P.hT[r] != nullptr ? marks.ends : 0u;
#pragma unroll
    for (int i = 0; i < kScanRun; ++i) {
      float y[2] = {through<PACKED>(f[i][0], h[i][0], in.x), through<PACKED>(f[i][1], h[i][1], in.y)};
      if ((ends >> i) & 1u) slot[i][lane] = make_float2(y[0], y[1]);
      if (on && tok0 + i < P.s) {
        Two<DT> o;
        pack(o, y);
        store_pack(out + (tok0 + i) * P.ld_out, o);
      }
    }
    put_states<PACKED>(P, P.hT[r], ends, tok0, bi, ch, on, slot);
  }
}

// One token a sequence: nothing to join.  Eight channels a thread.
template <int DT>
__global__ void __launch_bounds__(128) scan_step_kernel(const ScanParams P) {
  constexpr int E = ElemSize<DT>::value;
  pdl_wait();
  const int per = P.c / 8;
  const int64_t n = static_cast<int64_t>(P.b) * P.t * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = i / per;
    const int ch = static_cast<int>(i - row * per) * 8;
    const int r = static_cast<int>(row / P.b);
    const int64_t bi = row - static_cast<int64_t>(r) * P.b;
    Pack<DT, 8> graw, vraw, o;
    Pack<SP_F32, 8> h{};
    load_pack(graw, P.gate[r] + bi * P.ld_gate + static_cast<int64_t>(ch) * E);
    load_pack(vraw, P.value[r] + bi * P.ld_value + static_cast<int64_t>(ch) * E);
    if (P.h0[r] != nullptr)
      load_pack(h, reinterpret_cast<const char*>(P.h0[r] + bi * P.c + ch));
    float g[8], v[8], x[8];
    unpack(graw, g);
    unpack(vraw, v);
    unpack(h, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float a, k;
      gate_of<DT>(g[e], a, k);
      x[e] = P.tied ? fmaf(k, v[e] - x[e], x[e]) : fmaf(a, x[e], v[e]);
    }
    pack(o, x);
    store_pack(P.out[r] + bi * P.ld_out + static_cast<int64_t>(ch) * E, o);
    if (P.states[r] != nullptr) store_pack(reinterpret_cast<char*>(P.states[r] + bi * P.c + ch), h);
    if (P.hT[r] != nullptr) {
      pack(h, x);
      store_pack(reinterpret_cast<char*>(P.hT[r] + bi * P.c + ch), h);
    }
  }
}

void scan_shape(const ScanParams& p, int* warps, int* cluster) {
  const int64_t runs = (p.s + kScanRun - 1) / kScanRun;
  int w = 1;
  while (w < 8 && w < runs) w *= 2;
  const int64_t units = static_cast<int64_t>(p.slabs) * p.t * p.b;
  const int64_t want = 2 * static_cast<int64_t>(device_sm_count());
  int c = 1;
  while (c < kScanMaxCluster && units * c < want && static_cast<int64_t>(c) * w < runs) c *= 2;
  *warps = w;
  *cluster = c;
}

template <int DT>
static const void* scan_fwd_fn(bool tied, bool packed) {
  if (tied)
    return packed ? reinterpret_cast<const void*>(&scan_fwd_kernel<DT, true, true>)
                  : reinterpret_cast<const void*>(&scan_fwd_kernel<DT, true, false>);
  return packed ? reinterpret_cast<const void*>(&scan_fwd_kernel<DT, false, true>)
                : reinterpret_cast<const void*>(&scan_fwd_kernel<DT, false, false>);
}

cudaError_t launch_scan(const void* fn, const ScanParams& p, int warps, void** args,
                        cudaStream_t st) {
  const size_t smem = static_cast<size_t>(warps) * kScanRun * 32 * sizeof(float2);
  cudaError_t e = ensure_smem_attr(fn, smem);
  if (e == cudaSuccess && p.cluster > 8)
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  const int64_t blocks = static_cast<int64_t>(p.slabs) * p.t * p.b * p.cluster;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(fn, dim3(static_cast<unsigned>(blocks)), dim3(32 * warps), smem, args, st,
                    p.cluster);
}

cudaError_t launch_scan_fwd(ScanParams p, int dtype, cudaStream_t st) {
  void* args[] = {&p};
  const bool packed = p.cu_seqlens != nullptr;
  if (p.s == 1 && !packed) {
    const int64_t blocks = (static_cast<int64_t>(p.b) * p.t * (p.c / 8) + 127) / 128;
    const int64_t cap = static_cast<int64_t>(device_sm_count()) * 16;
    const void* fn = dtype == SP_BF16  ? reinterpret_cast<const void*>(&scan_step_kernel<SP_BF16>)
                     : dtype == SP_F16 ? reinterpret_cast<const void*>(&scan_step_kernel<SP_F16>)
                                       : reinterpret_cast<const void*>(&scan_step_kernel<SP_F32>);
    return launch_pdl(fn, dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)), dim3(128), 0,
                      args, st);
  }
  int warps;
  scan_shape(p, &warps, &p.cluster);
  const void* fn = dtype == SP_BF16  ? scan_fwd_fn<SP_BF16>(p.tied, packed)
                   : dtype == SP_F16 ? scan_fwd_fn<SP_F16>(p.tied, packed)
                                     : scan_fwd_fn<SP_F32>(p.tied, packed);
  return launch_scan(fn, p, warps, args, st);
}

}  // namespace spb
