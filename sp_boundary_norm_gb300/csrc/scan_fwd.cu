// Gated recurrence, forward: y, the last state of every sequence, and the
// state entering every run of 16 tokens for the backward.  One token of every
// sequence (a decoding step) takes a kernel without the joins.
#include <cmath>

#include "scan.cuh"

namespace spb {

// Blocks of up to four warps an SM that the registers are held to: three, or for dense
// 16-bit batches of many short sequences four, which spill a few registers (8192
// channels of 8 rows of 2048 tokens 139 us with three, 144 with four; 2048 of 16 rows of
// 1000 46 and 40, 512 of 64 rows of 100 8.9 and 6.8, 1024 of 300 rows of 33 37 and 32).
constexpr int kFwdBlocks = 3, kFwdMoreBlocks = 4;

// One run: h[i], f[i] with h[i] + f[i] * (state entering the run) the state
// after token i.  i0, h0: the first token that begins a sequence and the state
// before it; begin(i): that of any other.
template <int DT, bool TIED, int KIND, typename Shared, typename Begin>
__device__ __forceinline__ Map2 scan_run(const Shared& sh, int stage, uint32_t starts, int i0,
                                         F2 h0, F2 (&h)[kScanRun], F2 (&f)[kScanRun],
                                         Begin begin) {
  F2 cur = f2(0.f, 0.f);
  RunFactor fac;
#pragma unroll
  for (int i = 0; i < kScanRun; ++i) {
    if (KIND == kSingleRun && i == i0) {
      cur = h0;
      fac.cut();
    }
    if (KIND == kAnyRun && ((starts >> i) & 1u)) {
      cur = begin(i);
      fac.cut();
    }
    F2 e;
    const F2 a = open_gate<DT>(sh.template raw<DT>(stage, 0, i), e), k = mul2(e, a);
    cur = next_state<TIED>(a, k, cur, sh.template row<DT>(stage, 1, i));
    fac.next(a, k);
    h[i] = cur;
    f[i] = fac.a;
  }
  return Map2{fac.whole(), cur};
}

// BLOCKS: an SM's; 1: a wide block.
template <int DT, bool TIED, bool PACKED, int BLOCKS>
__global__ void __launch_bounds__(32 * (BLOCKS == 1 ? kScanWideWarps : kScanWarps), BLOCKS)
scan_fwd_kernel(const ScanParams P) {
  constexpr int E = ElemSize<DT>::value;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
  const int nw = blockDim.x >> 5;
  const int C = P.cluster, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const ScanShared<E, 2> sh(smem, warp, nw, C);
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
  const int64_t row0 = bi * P.s;
  const char* gate = P.gate[r] + row0 * P.ld_gate + static_cast<int64_t>(ch0) * E;
  const char* value = P.value[r] + row0 * P.ld_value + static_cast<int64_t>(ch0) * E;
  char* out = P.out[r] + row0 * P.ld_out + static_cast<int64_t>(ch) * E;
  const int64_t n_runs = (P.s + kScanRun - 1) / kScanRun;
  float* states = P.states[r];
  if (states != nullptr) states += bi * n_runs * P.c + ch;
  if (PACKED && rank == 0) pass_empty(P, P.h0[r], P.hT[r], ch, on);

  const int64_t stretch = static_cast<int64_t>(C) * nw * kScanRun;
  int64_t tok0 = static_cast<int64_t>(rank * nw + warp) * kScanRun;
  auto fetch = [&](int stage, int64_t at) {
    sh.copy(stage, 0, gate, P.ld_gate, at, P.s, bytes);
    sh.copy(stage, 1, value, P.ld_value, at, P.s, bytes);
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kStages; ++k) fetch(k, tok0 + k * stretch);
  F2 carry = f2(0.f, 0.f);
  SeqWindow win = no_window();
  int step = 0;
  int late = kNever;
  for (int64_t base = 0; base < P.s; base += stretch, tok0 += stretch, ++step) {
    const RunMarks marks = run_marks<PACKED>(P, tok0, win, sh.first, 0);
    const int kind = run_kind(marks, P.s - tok0);
    auto seq = [&](int i) { return seq_of_run<PACKED>(win, sh.first, marks.starts, bi, i); };
    auto begin = [&](int i) { return load_state(P.h0[r], seq(i), P.c, ch, on); };
    // (the first beginning's state is asked for beneath the wait for the rows)
    const int i0 = __ffs(marks.starts) - 1, i1 = 31 - __clz(marks.ends);
    F2 h0 = f2(0.f, 0.f);
    if (i0 >= 0) h0 = begin(i0);
    F2 h[kScanRun], f[kScanRun];
    sh.wait();
    const int stage = step % kStages;
    Map2 mine;
    if (kind == kPlainRun)
      mine = scan_run<DT, TIED, kPlainRun>(sh, stage, 0u, 0, h0, h, f, begin);
    else if (kind == kSingleRun)
      mine = scan_run<DT, TIED, kSingleRun>(sh, stage, 0u, i0, h0, h, f, begin);
    else
      mine = scan_run<DT, TIED, kAnyRun>(sh, stage, marks.starts, 0, h0, h, f, begin);
    __syncwarp();                     // every lane has read the rows
    fetch(stage, tok0 + kStages * stretch);
    const F2 entry = join_runs<PACKED, 1>(sh.join, step, mine, marks.starts != 0u, C, rank, warp, nw,
                                          P.withhold, carry, late);
    if (tok0 >= P.s) continue;
    if (states != nullptr && on)
      __stcs(reinterpret_cast<float2*>(states + (tok0 / kScanRun) * P.c), split(entry));
    char* at = out + tok0 * P.ld_out;
    if (kind == kPlainRun) {
      if (on) {
#pragma unroll
        for (int i = 0; i < kScanRun; ++i)
          store_pack(at + static_cast<uint64_t>(P.ld_out) * i, pack2<DT>(fma2(f[i], entry, h[i])));
      }
    } else if (kind == kSingleRun) {
      F2 last = f2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kScanRun; ++i) {
        // (from its beginning on a packed sequence has all of its state in h)
        const bool own = PACKED && static_cast<uint32_t>(i) >= static_cast<uint32_t>(i0);
        const F2 y = own ? h[i] : fma2(f[i], entry, h[i]);
        if (i == i1) last = y;
        if (on) store_pack(at + static_cast<uint64_t>(P.ld_out) * i, pack2<DT>(y));
      }
      if (i1 >= 0) store_state(P.hT[r], seq(i1), P.c, ch, on, last);
    } else {
      const int rows = P.s - tok0 < kScanRun ? static_cast<int>(P.s - tok0) : kScanRun;
#pragma unroll
      for (int i = 0; i < kScanRun; ++i) {
        const bool own = PACKED && (marks.starts & ((2u << i) - 1u)) != 0u;
        const F2 y = own ? h[i] : fma2(f[i], entry, h[i]);
        if ((marks.ends >> i) & 1u) store_state(P.hT[r], seq(i), P.c, ch, on, y);
        if (on && i < rows) store_pack(at + static_cast<uint64_t>(P.ld_out) * i, pack2<DT>(y));
      }
    }
  }
  cp_async_wait<0>();
  if (C > 1) leave_cluster<1>(sh.join, C, warp, nw, late, step, P.status);
}

// One token a sequence: nothing to join.  Eight channels a thread, 16-byte loads
// and stores.  64 sequences of 8 ranks of 1024 channels, 7.3 MB: 2.2 us, the launch
// and one trip to memory (at the copy rate the bytes take 1.1).
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
    float v[8], x[8];
    unpack(vraw, v);
    unpack(h, x);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      F2 e;
      Two<DT> g;
#pragma unroll
      for (int w = 0; w < Two<DT>::kWords; ++w) g.w[w] = graw.w[i / 2 * Two<DT>::kWords + w];
      F2 a = open_gate<DT>(g, e);
      const F2 k = mul2(e, a), minus = f2(-1.f, -1.f);
      // a without the reciprocal's error, a + a (1 - a - k): a kept state takes many steps
      a = fma2(a, fma2(k, minus, fma2(a, minus, f2(1.f, 1.f))), a);
      const F2 old = f2(x[i], x[i + 1]), val = f2(v[i], v[i + 1]);
      const float2 y = split(P.tied ? next_state<true>(a, k, old, val)
                                    : next_state<false>(a, k, old, val));
      x[i] = y.x;
      x[i + 1] = y.y;
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

template <int DT, bool TIED, bool PACKED>
static ScanKernels scan_fwd_kernels() {
  ScanKernels k{};
  k.fn = reinterpret_cast<const void*>(&scan_fwd_kernel<DT, TIED, PACKED, kFwdBlocks>);
  k.wide = reinterpret_cast<const void*>(&scan_fwd_kernel<DT, TIED, PACKED, 1>);
  if constexpr (!PACKED && DT != SP_F32)
    k.more = reinterpret_cast<const void*>(&scan_fwd_kernel<DT, TIED, false, kFwdMoreBlocks>);
  return k;
}
template <int DT>
static ScanKernels scan_fwd_kernels(bool tied, bool packed) {
  if (tied) return packed ? scan_fwd_kernels<DT, true, true>() : scan_fwd_kernels<DT, true, false>();
  return packed ? scan_fwd_kernels<DT, false, true>() : scan_fwd_kernels<DT, false, false>();
}

// Blocks of up to four warps, of which an SM takes several (lone ones of kernel `more`
// one more, each a tenth slower), or of 8 or 12 that have an SM to themselves (kernel
// `wide`); C blocks a cluster, for the split with the least expected time: the clusters that fit the GPU at once run in
// waves, and a step of a wave takes its shortest time and that of its bytes at
// 6.0 TB/s: a lone block's copies lie beneath its arithmetic and the longer one
// counts, a cluster's blocks wait for each other's (the cubes add up).  Many channels
// fill the GPU with lone or small blocks; few channels need long steps, because what a
// step costs grows less than its warps.  Measured, bf16, forward and backward in us:
//   16,384 tokens of 8192 channels: 4 warps, C = 1 213, 362; C = 3 164, 241; C = 4
//     200, 292; 12 warps, C = 1 151, 235; C = 2 197, 281
//   the same in 12 packed sequences: 4 warps, C = 3 190, 276; 12, C = 1 171, 263
//   8 rows of 2048 of 8192: 4 warps, C = 1 138, 236; C = 2 151, 236; 12, C = 1 149, 238
//   16,384 of 1024: 4 warps, C = 16 39, 55; 8, C = 12 51, 67; 12, C = 6 40, 55
//   65,537 of 512: 4 warps, C = 16 114, 162; 8, C = 12 89, 117; 12, C = 12 78, 107
cudaError_t launch_scan(const ScanKernels& kernels, ScanParams& p, int elem,
                        const ScanCost& cost, void** args, cudaStream_t st) {
  const int64_t runs = (p.s + kScanRun - 1) / kScanRun;
  const int64_t units = static_cast<int64_t>(p.slabs) * p.t * p.b;
  static const int kClusters[] = {1, 2, 3, 4, 6, 8, 12, kScanMaxCluster};
  int few = 1;
  while (few < kScanWarps && few < runs) few *= 2;
  const struct {
    const void* kernel;
    int warps, most;       // blocks of a cluster, at most
    double slower;
  } choices[] = {{kernels.fn, few, kScanMaxCluster, 1.0},
                 {kernels.more, few, 1, 1.1},
                 {kernels.wide, 8, kScanMaxCluster, 1.0},
                 {kernels.wide, kScanWideWarps, kScanMaxCluster, 1.0}};
  double best = 0;
  size_t smem = 0;
  int threads = 0;
  const void* chosen = nullptr;
  for (const auto& k : choices) {
    const int warps = k.warps;
    if (k.kernel == nullptr || (warps > kScanWarps && runs <= kScanWarps)) continue;
    for (const int c : kClusters) {
      if (c > k.most || (c > 1 && static_cast<int64_t>(c - 1) * warps >= runs)) break;
      const size_t need = scan_smem(elem, cost.tensors, warps, c);
      if (need > kScanMaxShared) break;
      const double bytes = static_cast<double>(c) * warps * kScanRun * kScanChannels * elem *
                           cost.passes;
      const double least = (c == 1 ? cost.lone : cost.cluster + c * cost.per_block) +
                           warps * cost.per_warp;
      const int64_t steps = (runs + static_cast<int64_t>(c) * warps - 1) / (c * warps);
      const double start = c == 1 ? 2.0 : 3.0;    // a wave's launch and first rows
      auto wave = [&](int64_t clusters) {
        const double moved = static_cast<double>(clusters) * bytes / 6.0e6;
        return start + k.slower * static_cast<double>(steps) *
                           (c == 1 ? (least > moved ? least : moved)
                                   : std::cbrt(least * least * least + moved * moved * moved));
      };
      if (smem != 0 && wave(0) >= best) continue;
      int fit = 0;
      const cudaError_t e = max_clusters(k.kernel, 32 * warps, need, c, &fit);
      if (e != cudaSuccess) return e;
      if (fit < 1) continue;
      const double time = static_cast<double>(units / fit) * wave(fit) +
                          (units % fit != 0 ? wave(units % fit) : 0.0);
      if (smem == 0 || time < best) {
        best = time;
        smem = need;
        threads = 32 * warps;
        chosen = k.kernel;
        p.cluster = c;
      }
    }
  }
  if (smem == 0 || units * p.cluster > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(chosen, dim3(static_cast<unsigned>(units * p.cluster)), dim3(threads), smem,
                    args, st, p.cluster);
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
  const ScanKernels kernels = dtype == SP_BF16  ? scan_fwd_kernels<SP_BF16>(p.tied, packed)
                              : dtype == SP_F16 ? scan_fwd_kernels<SP_F16>(p.tied, packed)
                                                : scan_fwd_kernels<SP_F32>(p.tied, packed);
  const ScanCost cost = dtype == SP_F32 ? ScanCost{0.2, 0.53, 0.03, 0.19, 2, 3}
                                        : ScanCost{0.26, 0.64, 0.038, 0.125, 2, 3};
  return launch_scan(kernels, p, dtype == SP_F32 ? 4 : 2, cost, args, st);
}

}  // namespace spb
