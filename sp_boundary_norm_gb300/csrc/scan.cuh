// Shared parts of the gated recurrence's forward and backward:
//   a = sigmoid(gate), k = sigmoid(-gate) = 1 - a
//   h[i] = a[i] h[i-1] + k[i] v[i]   (tied)   or   a[i] h[i-1] + v[i]   (free)
// along the tokens of a sequence, each channel on its own.
//
// A block takes 64 channels, two a lane, and 16 tokens a warp (a "run"): a
// thread scans its run in registers and knows it as an affine map h -> A h + H.
// The maps are joined over the block's warps in shared memory and over the
// blocks of a cluster by asynchronous stores into every block's shared memory,
// always in token order, so results do not depend on timing; then the cluster
// steps to the next stretch of the sequence with the state in registers.  The
// next stretch's rows are on their way (16-byte cp.async, four rows an
// instruction) from the moment the present ones are in registers.  Nothing is
// read twice and no block waits for another but its cluster's.
//
// Measured on a GB300, bf16 (the rate is of the bytes that have to move; the
// measured copy rate is 6.8 TB/s): 8 ranks of 16,384 tokens x 1024 channels,
// forward 151 us (5.3 TB/s), backward 235 (5.7); packed as 12 sequences
// 171 and 263; 1 rank of 65,537 x 512 77 and 107, where the steps' joins are what
// takes time: few channels cannot fill the SMs otherwise.
//
// Two exponentials' worth of special functions, a scan and a correction an
// element sit between 6 and 10 bytes of traffic, so instructions count as much
// as bytes: the two channels of a lane go through packed float32 arithmetic,
// and whole runs inside one sequence take code without its checks.
#pragma once

#include "region.cuh"

namespace spb {

// Two channels of one token.
template <int DT>
using Two = Pack<DT, 2>;

template <int DT>
__device__ __forceinline__ F2 unpack2(const Two<DT>& p) {
  float f[2];
  unpack(p, f);
  return f2(f[0], f[1]);
}
template <int DT>
__device__ __forceinline__ Two<DT> pack2(F2 v) {
  const float2 f = split(v);
  const float w[2] = {f.x, f.y};
  Two<DT> p;
  pack(p, w);
  return p;
}

// Two gates held above -87, where exp(-g) and its reciprocal are normal numbers (16-bit
// types: both at once; exp2_of does it for float32).  NaN stays NaN.
template <int DT>
__device__ __forceinline__ Two<DT> held_gate(Two<DT> g) {
  if constexpr (DT == SP_BF16) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(g.w[0]) : "r"(0xC2AEC2AEu));
  if constexpr (DT == SP_F16) asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(g.w[0]) : "r"(0xD570D570u));
  return g;
}

// a = sigmoid(g) = 1 / (1 + e) from e = exp(-g), and k = e a: both keep their
// relative digits however small they are.  (1 - k in place of a, as in h + k (v - h),
// is off by 2^-24: all of a shut gate's a, which is what is left of a state that
// gathered over thousands of tokens.)  Gates below -87 count as -87: a = 2^-126, and so
// does k of gates above 87, which is flushed to 0.
template <int DT>
__device__ __forceinline__ F2 open_gate(Two<DT> g, F2& e) {
  e = exp2_of<DT, DT == SP_F32, -1>(unpack2<DT>(held_gate<DT>(g)));
  return rcp2(add2(e, f2(1.f, 1.f)));
}

// The state after a token: a h + k v, or a h + v.
template <bool TIED>
__device__ __forceinline__ F2 next_state(F2 a, F2 k, F2 h, F2 v) {
  return fma2(a, h, TIED ? mul2(k, v) : v);
}

// The product of the a of a run, and 1 - that product, a sum of k a...a.  An open gate's
// a, next to 1, is off by up to 2^-23, and products of such numbers round to one side:
// over a memory of 1/k tokens that adds up (65,537 tokens with k around 1e-5: 2e-5 of
// the state, against 2e-6).  So what passes from run to run is 1 - lost while that is at
// least 1/2; the product, which has the digits of shut gates, otherwise and in the run.
struct RunFactor {
  F2 a = f2(1.f, 1.f), lost = f2(0.f, 0.f);
  __device__ __forceinline__ void next(F2 ai, F2 ki) {
    lost = fma2(a, ki, lost);
    a = mul2(a, ai);
  }
  __device__ __forceinline__ void cut() {
    a = f2(0.f, 0.f);
    lost = f2(1.f, 1.f);
  }
  __device__ __forceinline__ F2 whole() const {
    const float2 x = split(a), y = split(lost);
    return f2(y.x <= 0.5f ? 1.f - y.x : x.x, y.y <= 0.5f ? 1.f - y.y : x.y);
  }
};

// The affine maps of a thread's two channels over some tokens: x -> a x + h.
struct alignas(16) Map2 {
  F2 a, h;
};

// The map's value at x.  CUT (packed batches): a sequence that begins inside the map's
// tokens cuts off what comes before them, and what x holds (an infinity, a NaN) must
// not pass.  A factor of zero says so, and nothing else does: a product of a's that
// underflows inside a sequence counts as 2^-149, so that what is not finite there stays.
template <bool CUT>
__device__ __forceinline__ F2 through(F2 a, F2 h, F2 x) {
  const F2 y = fma2(a, x, h);
  if constexpr (!CUT) return y;
  const float2 f = split(a), g = split(h), w = split(y);
  return f2(f.x == 0.f ? g.x : w.x, f.y == 0.f ? g.y : w.y);
}

constexpr float kLeast = 0x1p-149f;
__device__ __forceinline__ float at_least(float v, float least) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(least));
  return v;
}
// The factor of a run's map: zero only for a cut.
__device__ __forceinline__ F2 uncut(F2 a) {
  const float2 v = split(a);
  return f2(at_least(v.x, kLeast), at_least(v.y, kLeast));
}
// The factor of map a after map b: zero only if either's is, and if a's is, whatever b's.
__device__ __forceinline__ F2 uncut_product(F2 a, F2 b) {
  const float2 v = split(a), w = split(b), p = split(mul2(a, b));
  return f2(v.x == 0.f ? 0.f : at_least(p.x, fminf(w.x, kLeast)),
            v.y == 0.f ? 0.f : at_least(p.y, fminf(w.y, kLeast)));
}

// Map m into the cluster address `to`, counted in bytes on the mbarrier `bar`
// (also a cluster address) of the same block.
__device__ __forceinline__ void st_async_map(uint32_t to, const Map2& m, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(
          to),
      "l"(m.a), "l"(m.h), "r"(bar)
      : "memory");
}

// Which of the run's tokens tok0 .. tok0 + 15 begin a sequence, and which end one.
struct RunMarks {
  uint32_t starts, ends;
};

// What a warp knows of a packed batch: 32 consecutive entries of cu_seqlens, one
// a lane, and of the sequence that its last marked run began in the tokens
// [lo, hi).  Runs inside it take two comparisons, others within the entries a
// few votes; only the rest go back to memory.
struct SeqWindow {
  int base, at;        // first entry; this lane's (INT_MAX behind the last)
  int seq, lo, hi;
};

__device__ __forceinline__ SeqWindow no_window() { return SeqWindow{0, 0x7FFFFFFF, 0, 0, 0}; }

// `first`: 16 words of the warp's shared memory, set for every start bit to the
// sequence that begins there (the last of several: the others are empty).
// `back`: entries to keep before the run's (a walk towards the beginning).
template <bool PACKED>
__device__ __forceinline__ RunMarks run_marks(const ScanParams& P, int64_t tok0, SeqWindow& win,
                                              int* first, int back) {
  if (tok0 >= P.s) return RunMarks{0u, 0u};
  // bit i: token tok0 + i is the first of a sequence, or the first after the call's last
  uint32_t m = tok0 == 0 ? 1u : 0u;
  if constexpr (PACKED) {
    const int tok = static_cast<int>(tok0), n = P.n_seqs;
    if (tok <= win.lo || static_cast<int64_t>(tok) + kScanRun >= win.hi) {
      const int lane = threadIdx.x & 31;
      const int end = P.s - tok0 > kScanRun ? tok + kScanRun : static_cast<int>(P.s - 1);
      const int w0 = __shfl_sync(0xFFFFFFFFu, win.at, 0), w31 = __shfl_sync(0xFFFFFFFFu, win.at, 31);
      if (w0 > tok || w31 <= end) {
        const int j = seq_of_token(P.cu_seqlens, n, tok0);
        win.base = j > back ? j - back : 0;
        win.at = win.base + lane <= n ? __ldg(P.cu_seqlens + win.base + lane) : 0x7FFFFFFF;
      }
      const uint32_t le = __ballot_sync(0xFFFFFFFFu, win.at <= tok && win.base + lane < n);
      const int k = le != 0u ? 31 - __clz(le) : 0;
      win.seq = win.base + k;
      win.lo = __shfl_sync(0xFFFFFFFFu, win.at, k);
      win.hi = __shfl_sync(0xFFFFFFFFu, win.at, k < 31 ? k + 1 : 31);
      __syncwarp();                   // every lane is done with the run before
      if (lane < kScanRun) first[lane] = win.seq;
      __syncwarp();
      for (int j = win.base; j < n; j += 32) {     // one round unless 32 sequences begin here
        const int at = j == win.base ? win.at
                       : j + lane < n ? __ldg(P.cu_seqlens + j + lane) : 0x7FFFFFFF;
        const bool in = at >= tok && at <= end && j + lane < n;
        m |= __reduce_or_sync(0xFFFFFFFFu, in ? 1u << (at - tok) : 0u);
        if (in && at - tok < kScanRun) atomicMax(first + (at - tok), j + lane);
        if (__any_sync(0xFFFFFFFFu, at > end)) break;
      }
      __syncwarp();
    }
  }
  const int left = P.s - tok0 <= kScanRun ? static_cast<int>(P.s - tok0) : kScanRun + 1;
  const uint32_t starts = m & ((1u << (left < kScanRun ? left : kScanRun)) - 1u);
  if (left <= kScanRun) m |= 1u << left;
  return RunMarks{starts, (m >> 1) & 0xFFFFu};
}

// The sequence of the run's token i.
template <bool PACKED>
__device__ __forceinline__ int seq_of_run(const SeqWindow& win, const int* first, uint32_t starts,
                                          int bi, int i) {
  if constexpr (!PACKED) return bi;
  const uint32_t m = starts & ((2u << i) - 1u);
  return m != 0u ? first[31 - __clz(m)] : win.seq;
}

// A thread's two channels (from `ch`) of a sequence's state; NULL = zeros.  (Not
// inlined: a run with several marks asks for them from many places.)
static __device__ __noinline__ F2 load_state(const float* src, int seq, int c, int ch, bool on) {
  if (src == nullptr || !on) return f2(0.f, 0.f);
  const float2 v = *reinterpret_cast<const float2*>(src + static_cast<int64_t>(seq) * c + ch);
  return f2(v.x, v.y);
}
static __device__ __noinline__ void store_state(float* dst, int seq, int c, int ch, bool on, F2 v) {
  if (dst != nullptr && on)
    *reinterpret_cast<float2*>(dst + static_cast<int64_t>(seq) * c + ch) = split(v);
}

// What a run has to look out for: nothing (whole and inside one sequence); at
// most one beginning and one end, all 16 tokens there (their states come in
// registers); anything.
constexpr int kPlainRun = 0, kSingleRun = 1, kAnyRun = 2;

__device__ __forceinline__ int run_kind(const RunMarks& m, int64_t left) {
  if ((m.starts | m.ends) == 0u) return kPlainRun;
  return __popc(m.starts) <= 1 && __popc(m.ends) <= 1 && left >= kScanRun ? kSingleRun : kAnyRun;
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

// Joins the runs' maps in token order (TIME = +1) or against it (-1): from the
// value that enters the cluster's stretch (`carry`, which moves behind the
// stretch) the value that enters this thread's run, whose map is `mine`; `cut`: a
// sequence begins (ends) in the run.
//
// The maps of a block meet in `run`; a warp folds those before its own, and the
// last one's fold, the block's map, goes to every block of the cluster by
// asynchronous stores that count their bytes on the receiver's mbarrier.
// Buffers and mbarriers alternate between two; a block's map of step n + 2 is
// sent after all maps of step n + 1 have arrived, which their blocks sent after
// they had read step n's, so nothing is overwritten before it is read.
//
// The wait is bounded: `late` is the step in which a thread's ran out (kNever), and it
// waits no more.  The warp that sends the block's map also arms (lane 0) the mbarriers
// for the partners' maps, one step after the other; a late lane does neither, so its
// partners' waits run out too, and no mbarrier is armed again before its phase is over.
struct JoinBuffers {
  Map2* run;        // [2][warps][32]
  Map2* block;      // [2][cluster][32]
  uint64_t* bar;    // [2]
};
constexpr int kNever = 0x7FFFFFFF;

constexpr int kFold = 4;    // maps read at once
constexpr int kStages = 2;  // runs of a warp on their way

// The value x taken through n maps (`at`: this lane's of the first one in
// time; `step` from one to the next); *in: the value before map `place`.
template <bool CUT>
__device__ __forceinline__ F2 fold_value(const Map2* at, int step, int n, int place, F2 x, F2* in) {
  for (int k0 = 0; k0 < n; k0 += kFold) {
    Map2 m[kFold];
#pragma unroll
    for (int u = 0; u < kFold; ++u)
      if (k0 + u < n) m[u] = at[(k0 + u) * step];
#pragma unroll
    for (int u = 0; u < kFold; ++u) {
      if (k0 + u == place) *in = x;
      if (k0 + u < n) x = through<CUT>(m[u].a, m[u].h, x);
    }
  }
  return x;
}

// Map `acc` followed by map m.
template <bool CUT>
__device__ __forceinline__ void fold_map(Map2& acc, const Map2& m) {
  acc.h = through<CUT>(m.a, m.h, acc.h);
  acc.a = CUT ? uncut_product(m.a, acc.a) : mul2(m.a, acc.a);
}
template <bool CUT>
__device__ __forceinline__ Map2 fold_maps(const Map2* at, int step, int n) {
  Map2 acc{f2(1.f, 1.f), f2(0.f, 0.f)};
  for (int k0 = 0; k0 < n; k0 += kFold) {
    Map2 m[kFold];
#pragma unroll
    for (int u = 0; u < kFold; ++u)
      if (k0 + u < n) m[u] = at[(k0 + u) * step];
#pragma unroll
    for (int u = 0; u < kFold; ++u)
      if (k0 + u < n) fold_map<CUT>(acc, m[u]);
  }
  return acc;
}

template <bool CUT, int TIME>
__device__ __forceinline__ F2 join_runs(const JoinBuffers& sh, int step, Map2 mine, bool cut,
                                        int C, int rank, int warp, int nw, int withhold,
                                        F2& carry, int& late) {
  if (CUT && !cut) mine.a = uncut(mine.a);
  const int lane = threadIdx.x & 31;
  const int par = step & 1;
  Map2* run = sh.run + par * nw * 32 + lane;
  run[warp * 32] = mine;
  const int place = TIME > 0 ? warp : nw - 1 - warp;
  const bool sends = place == nw - 1 && late == kNever;
  if (C > 1 && sends && lane == 0) mbar_arrive_expect_tx(&sh.bar[par], C * 32 * sizeof(Map2));
  __syncthreads();
  const Map2* run0 = TIME > 0 ? run : run + (nw - 1) * 32;
  F2 in = carry;
  if (C == 1) {
    // values in place of maps: the carry is known
    carry = fold_value<CUT>(run0, TIME * 32, nw, place, carry, &in);
    return in;
  }
  const Map2 before = fold_maps<CUT>(run0, TIME * 32, place);
  Map2* block = sh.block + par * C * 32 + lane;
  if (sends && !(blockIdx.x == 0 && step == withhold)) {
    Map2 all = before;
    fold_map<CUT>(all, mine);
    for (int peer = 0; peer < C; ++peer)
      st_async_map(cluster_map(block + rank * 32, peer), all, cluster_map(&sh.bar[par], peer));
  }
  if (late == kNever && !mbar_wait_cluster(&sh.bar[par], (step >> 1) & 1)) late = step;
  const int place_c = TIME > 0 ? rank : C - 1 - rank;
  const Map2* block0 = TIME > 0 ? block : block + (C - 1) * 32;
  carry = fold_value<CUT>(block0, TIME * 32, C, place_c, carry, &in);
  return through<CUT>(before.a, before.h, in);
}

// The end of a cluster's blocks, of `steps` steps each.  Where the arming lane is late,
// partners' maps may still be on their way here: of the step it was late in, and of the
// next one, which partners go into that had all maps of the first (no further: they
// miss this block's).  Both are waited for, again with a limit.  (Where it is not, all
// maps of all steps are here.)
template <int TIME>
__device__ __forceinline__ void leave_cluster(const JoinBuffers& sh, int C, int warp, int nw,
                                              int late, int steps, int32_t* status) {
  cluster_sync_all();                          // no partner sends any more
  if (late == kNever) return;
  if (status != nullptr) *status = SP_ERR_TIMEOUT;
  if (warp != (TIME > 0 ? nw - 1 : 0) || (threadIdx.x & 31) != 0) return;
  const int next = late + 1;
  if (next < steps) mbar_arrive_expect_tx(&sh.bar[next & 1], C * 32 * sizeof(Map2));
  for (int step = late; step <= next && step < steps; ++step)
    mbar_wait_cluster(&sh.bar[step & 1], (step >> 1) & 1);
}

// The shared memory of a block: the ring of `tensors` inputs' runs, the joins'
// buffers and mbarriers, the runs' sequences.
__host__ __device__ constexpr size_t scan_smem(int elem, int tensors, int warps, int cluster) {
  return static_cast<size_t>(warps) * (32 * (static_cast<size_t>(kStages) * tensors * kScanRun * 2 *
                                                 elem + 2 * sizeof(Map2)) +
                                       kScanRun * sizeof(int)) +
         static_cast<size_t>(cluster) * 64 * sizeof(Map2) + 2 * sizeof(uint64_t);
}

template <int E, int TENSORS>
struct ScanShared {
  char* ring;                // this warp's rows
  int* first;                // sequences that begin in this warp's run
  JoinBuffers join;
  static constexpr int kRow = kScanChannels * E;      // bytes of a row piece
  static constexpr int kTensor = kScanRun * kRow;
  static constexpr int kStage = TENSORS * kTensor;
  // Called by every thread; the caller synchronises the block (or cluster).
  __device__ __forceinline__ ScanShared(char* base, int warp, int nw, int C) {
    ring = base + warp * kStages * kStage;
    base += nw * kStages * kStage;
    join.run = reinterpret_cast<Map2*>(base);
    join.block = join.run + 2 * nw * 32;
    base = reinterpret_cast<char*>(join.block + 2 * C * 32);
    join.bar = reinterpret_cast<uint64_t*>(base);
    first = reinterpret_cast<int*>(join.bar + 2) + warp * kScanRun;
    if (threadIdx.x == 0) {
      mbar_init(&join.bar[0], 1);
      mbar_init(&join.bar[1], 1);
      mbar_fence_init();
    }
  }
  template <int DT>
  __device__ __forceinline__ Two<DT> raw(int stage, int tensor, int i) const {
    const char* at = ring + stage * kStage + tensor * kTensor + i * kRow + (threadIdx.x & 31) * 2 * E;
    Two<DT> p;
    if constexpr (E == 4) {
      const uint2 v = lds8(at);
      p.w[0] = v.x;
      p.w[1] = v.y;
    } else {
      p.w[0] = *reinterpret_cast<const uint32_t*>(at);
    }
    return p;
  }
  template <int DT>
  __device__ __forceinline__ F2 row(int stage, int tensor, int i) const {
    return unpack2<DT>(raw<DT>(stage, tensor, i));
  }
  // Starts the copies into a stage of rows tok0 .. tok0 + 15 of a tensor (`src`: this slab's
  // first channel of token 0), zeros for rows and channels that do not exist.
  // `bytes`: of the slab's row pieces.
  __device__ __forceinline__ void copy(int stage, int tensor, const char* src, uint32_t ld, int64_t tok0,
                                       int64_t s, int bytes) const {
    constexpr int kLanes = kRow / 16, kRows = 32 / kLanes;    // lanes a row, rows at once
    const int lane = threadIdx.x & 31, col = lane % kLanes * 16, row0 = lane / kLanes;
    const uint32_t to = smem_addr(ring) + stage * kStage + tensor * kTensor + row0 * kRow + col;
    const int rows = col >= bytes || tok0 >= s || tok0 < 0 ? 0
                     : s - tok0 < kScanRun ? static_cast<int>(s - tok0) : kScanRun;
    const char* at = src + (rows > 0 ? tok0 * ld + col : 0);
#pragma unroll
    for (int i = 0; i < kScanRun / kRows; ++i) {
      const int row = row0 + i * kRows;
      const bool ok = row < rows;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * kRows * kRow),
                   "l"(at + static_cast<uint64_t>(ok ? row : 0) * ld), "r"(ok ? 16 : 0)
                   : "memory");
    }
  }
  // The oldest stage's copies are there for every lane.
  __device__ __forceinline__ void wait() const {
    cp_async_wait<kStages - 1>();
    __syncwarp();
  }
};

// How a direction's time depends on the split of a call, measured on a GB300
// in microseconds: the shortest step of a lone block, and of a cluster of C
// (cluster + C per_block), plus per_warp for each warp of a block; its tensors
// read, and read or written.
struct ScanCost {
  double lone, cluster, per_block, per_warp;
  int tensors, passes;
};

// A direction's kernels: small blocks, the same with one block an SM more (or NULL),
// blocks that have an SM to themselves.
struct ScanKernels {
  const void *fn, *more, *wide;
};

// Chooses the split of a call and launches its kernel.
cudaError_t launch_scan(const ScanKernels& kernels, ScanParams& p, int elem,
                        const ScanCost& cost, void** args, cudaStream_t st);

}  // namespace spb
