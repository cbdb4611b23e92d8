// Selective scan: a block's walk along its tokens, forward and, for the gradients'
// carries, backward.
//
// A block takes 32 channels of one rank's group (16 of 64 states) and walks its chunk
// of a batch row, 32 tokens a step.  The next steps' rows are on their way by 16-byte
// asynchronous copies; B and C become float32 in shared memory once for the block's
// warps, one step ahead; everything else is a warp's own: a lane prepares one token of
// the warp's channels (softplus, d u) into shared memory, the lanes then walk the 32
// tokens with their states in registers, and a lane finishes one token's outputs.  So
// the block meets once a step.
#include "ssm.cuh"

namespace spb {

// What a walk is for.
constexpr int kSsmOut = 0;     // y, and the states
constexpr int kSsmEnds = 1;    // a chunk's last state from a zero one, the sum of its steps
constexpr int kSsmBack = 2;    // a chunk's gradient for the state before it, from a zero
                               // one, and the sum of its steps

template <int DT, int N>
struct SsmWalk {
  using L = SsmLanes<N>;
  static constexpr int kWarps = N >= 32 ? 8 : 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kBlocks = kWarps == 8 ? 2 : 3;          // of an SM, by their registers
  static constexpr int kBlockCh = kWarps * L::kChannels;
  static constexpr int E = ElemSize<DT>::value;
  static constexpr int kStages = 3;
  // bytes: 16 more a row than it holds, so that lanes of different rows use
  // different banks
  static constexpr int kRow = kBlockCh * E + 16;
  static constexpr int kShared = 2 * N * E;                    // B and C of a token
  static constexpr int kStage = kSsmTile * (3 * kRow + kShared);
  static constexpr int kBC = kSsmTile * 2 * N * 4;             // float32 B and C
  static constexpr int kDRow = L::kChannels * 16 + 16;         // d, d, d u, d u a channel
  static constexpr int kYRow = L::kChannels * 4 + 16;
  static constexpr int kOwn = kSsmTile * (kDRow + kYRow);      // of a warp
  static constexpr int kParam = kBlockCh * 2 * 4;              // dt_bias and D
  static constexpr size_t kSmem = kStages * kStage + 2 * kBC + kWarps * kOwn + kParam;
};

template <int DT, int N, int MODE>
__global__ void __launch_bounds__(SsmWalk<DT, N>::kThreads, SsmWalk<DT, N>::kBlocks)
ssm_walk_kernel(const SsmParams P) {
  using W = SsmWalk<DT, N>;
  using L = SsmLanes<N>;
  constexpr int E = W::E, K = L::kPairs, CW = L::kChannels, G = L::kLanes, T = kSsmTile;
  constexpr bool kBack = MODE == kSsmBack;
  extern __shared__ __align__(16) char smem[];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (MODE != kSsmBack && blockIdx.x == 0 && warp == 0)
    check_cu_seqlens(P.cu_seqlens, P.n_seqs, P.s, P.status);
  const SsmPlace<W::kBlockCh> at(P);
  const int r = at.r;
  const int64_t rc = static_cast<int64_t>(r) * P.c;            // the rank's first channel
  char* bc = smem + W::kStages * W::kStage;
  char* own = bc + 2 * W::kBC + warp * W::kOwn;
  char* ybuf = own + T * W::kDRow;
  float* param = reinterpret_cast<float*>(bc + 2 * W::kBC + W::kWarps * W::kOwn);
  for (int i = tid; i < W::kBlockCh; i += W::kThreads) {
    const bool on = i < at.live;
    param[i] = on && P.dt_bias != nullptr ? P.dt_bias[rc + at.ch0 + i] : 0.f;
    param[W::kBlockCh + i] = on && P.D != nullptr ? P.D[rc + at.ch0 + i] : 0.f;
  }
  // the rows that a walk reads: dt, u (back: dy), z (not for ends); B (back: C), and C
  const int64_t row0 = at.batch * P.s + at.tok0;
  const char* src[3] = {P.dt[r] + row0 * P.ld_dt + at.ch0 * E,
                        (kBack ? P.dy[r] + row0 * P.ld_dy : P.u[r] + row0 * P.ld_u) + at.ch0 * E,
                        P.gated ? P.z[r] + row0 * P.ld_z + at.ch0 * E : nullptr};
  const int64_t lds[3] = {P.ld_dt, kBack ? P.ld_dy : P.ld_u, P.ld_z};
  const char* src_b = (kBack ? P.C[r] + row0 * P.ld_C : P.B[r] + row0 * P.ld_B) + at.group * N * E;
  const char* src_c = P.C[r] + row0 * P.ld_C + at.group * N * E;
  const int64_t ld_b = kBack ? P.ld_C : P.ld_B;
  const bool gated = MODE != kSsmEnds && P.gated;
  const int n_tiles = static_cast<int>((at.len + T - 1) / T);
  const int live_bytes = at.live * E;
  // step k's tile, in the order of the walk
  auto tile_of = [&](int k) { return static_cast<int64_t>(kBack ? n_tiles - 1 - k : k) * T; };
  auto ask = [&](int k) {
    char* st = smem + (k % W::kStages) * W::kStage;
    const int64_t t0 = tile_of(k);
    const int n_tok = at.len - t0 < T ? static_cast<int>(at.len - t0) : T;
    constexpr int kPieces = W::kBlockCh * E / 16;
#pragma unroll
    for (int i = tid; i < T * kPieces; i += W::kThreads) {
      const int tok = i / kPieces, p = (i % kPieces) * 16;
      if (tok >= n_tok || p >= live_bytes) continue;
      char* dst = st + tok * W::kRow + p;
      cp_async16(dst, src[0] + (t0 + tok) * lds[0] + p);
      cp_async16(dst + T * W::kRow, src[1] + (t0 + tok) * lds[1] + p);
      if (gated) cp_async16(dst + 2 * T * W::kRow, src[2] + (t0 + tok) * lds[2] + p);
    }
    constexpr int kP = N * E / 16;
    char* sh = st + 3 * T * W::kRow;
    for (int i = tid; i < n_tok * kP; i += W::kThreads) {
      const int tok = i / kP, p = (i - tok * kP) * 16;
      cp_async16(sh + tok * W::kShared + p, src_b + (t0 + tok) * ld_b + p);
      if (MODE == kSsmOut) cp_async16(sh + tok * W::kShared + N * E + p, src_c + (t0 + tok) * P.ld_C + p);
    }
  };
  // step k's B and C to float32
  auto widen = [&](int k) {
    const char* sh = smem + (k % W::kStages) * W::kStage + 3 * T * W::kRow;
    float* dst = reinterpret_cast<float*>(bc + (k & 1) * W::kBC);
    constexpr int kAll4 = T * 2 * N / 4;
    for (int i = tid; i < kAll4; i += W::kThreads) {
      if (MODE != kSsmOut && (i * 4) % (2 * N) >= N) continue;
      Pack<DT, 4> p;
      float f[4];
      lds_pack(p, sh + i * 4 * E);
      unpack(p, f);
      *reinterpret_cast<float4*>(dst + i * 4) = make_float4(f[0], f[1], f[2], f[3]);
    }
  };

  const bool active = warp * CW < at.live;
  const int n0 = (lane % G) * L::kStates, ch = warp * CW + lane / G;   // of the block
  // this lane's states: of [t * c][n], and of a rank's [sequences][c][n]
  const int64_t mine = (rc + at.ch0 + ch) * N + n0;
  const int64_t state_at = static_cast<int64_t>(at.ch0 + ch) * N + n0;
  const int64_t state_step = static_cast<int64_t>(P.c) * N;
  const int64_t carry_at = (at.batch * P.chunks + at.chunk) * P.t * P.c * N + mine;
  const bool packed = P.cu_seqlens != nullptr;
  F2 a2[K], h[K];
  int cur = -1;                        // the packed sequence that the state belongs to
  int64_t known = 0;                   // packed: no sequence begins in [tile, known)
  clear(h);
  clear(a2);
  if (active) {
    load_states(P.A + mine, a2);
#pragma unroll
    for (int p = 0; p < K; ++p) a2[p] = mul2(a2[p], f2(kLog2e, kLog2e));
    if constexpr (MODE == kSsmOut) {
      if (P.chunks > 1) load_states(P.carry + carry_at, h);
      else if (!packed) load_states_or_zero(P.h0[r], at.batch * state_step + state_at, h);
    }
    if (packed && at.tok0 > 0) cur = find_seq(P.cu_seqlens, P.n_seqs, at.tok0 - 1);
    if (packed && MODE == kSsmOut && at.chunk == 0 && P.hT[r] != nullptr &&
        P.hT[r] != P.h0[r]) {
      // the states of sequences without a token pass
      for (int j = 0; j < P.n_seqs; ++j) {
        if (__ldg(P.cu_seqlens + j) != __ldg(P.cu_seqlens + j + 1)) continue;
        F2 v[K];
        load_states_or_zero(P.h0[r], j * state_step + state_at, v);
        store_states(P.hT[r] + j * state_step + state_at, v);
      }
    }
  }
  float sum = 0.f;                     // of the chunk's steps

  if (n_tiles > 0) ask(0);
  cp_async_commit();
  if (n_tiles > 1) ask(1);
  cp_async_commit();
  cp_async_wait<1>();
  __syncthreads();
  if (n_tiles > 0) widen(0);
  for (int k = 0; k < n_tiles; ++k) {
    cp_async_wait<0>();
    __syncthreads();                   // step k + 1's rows, step k's B and C are there
    if (k + 2 < n_tiles) ask(k + 2);
    cp_async_commit();
    if (k + 1 < n_tiles) widen(k + 1);
    if (!active) continue;
    const char* st = smem + (k % W::kStages) * W::kStage + warp * CW * E;
    const float* shared = reinterpret_cast<const float*>(bc + (k & 1) * W::kBC);
    const int64_t t0 = tile_of(k), tok0 = at.tok0 + t0;
    const int n_tok = at.len - t0 < T ? static_cast<int>(at.len - t0) : T;

    // a lane's token: d and d u (back: silu(z) dy) of the warp's channels
    __syncwarp();
    {
      Pack<DT, CW> p;
      F2 d[CW / 2], v[CW / 2];
      lds_pack(p, st + lane * W::kRow);
      unpack_pairs(p, d);
      lds_pack(p, st + (T + lane) * W::kRow);
      unpack_pairs(p, v);
#pragma unroll
      for (int i = 0; i < CW / 2; ++i) {
        const float2 bias = *reinterpret_cast<const float2*>(param + warp * CW + 2 * i);
        d[i] = add2(d[i], f2(bias.x, bias.y));
        if (P.softplus) d[i] = softplus2<DT>(d[i], nullptr);
        if constexpr (!kBack) v[i] = mul2(d[i], v[i]);
      }
      if (kBack && gated) {
        F2 z[CW / 2];
        lds_pack(p, st + (2 * T + lane) * W::kRow);
        unpack_pairs(p, z);
#pragma unroll
        for (int i = 0; i < CW / 2; ++i)
          v[i] = mul2(v[i], mul2(z[i], rcp2(add2(exp2_of<DT, false, -1>(z[i]), f2(1.f, 1.f)))));
      }
#pragma unroll
      for (int i = 0; i < CW / 2; ++i) {
        const float2 a = split(d[i]), b = split(v[i]);
        float4* dst = reinterpret_cast<float4*>(own + lane * W::kDRow) + 2 * i;
        dst[0] = make_float4(a.x, a.x, b.x, b.x);
        dst[1] = make_float4(a.y, a.y, b.y, b.y);
      }
    }
    __syncwarp();

    // one token of a lane's states; the lane's part of its channel's sum with C
    float steps = 0.f;
    auto token = [&](int t) {
      const float4 d = *reinterpret_cast<const float4*>(own + t * W::kDRow + (lane / G) * 16);
      const F2 step = f2(d.x, d.y), in = f2(d.z, d.w);
      F2 b[K];
      load_states(shared + t * 2 * N + n0, b);
      if constexpr (MODE != kSsmOut) steps += d.x;
      if constexpr (kBack) {
#pragma unroll
        for (int p = 0; p < K; ++p) h[p] = mul2(pow2(mul2(step, a2[p])), fma2(in, b[p], h[p]));
        return 0.f;
      } else {
#pragma unroll
        for (int p = 0; p < K; ++p) h[p] = fma2(pow2(mul2(step, a2[p])), h[p], mul2(in, b[p]));
        if constexpr (MODE == kSsmEnds) return 0.f;
        F2 c[K];
        load_states(shared + t * 2 * N + N + n0, c);
        F2 acc = mul2(h[0], c[0]);
        if constexpr (K == 2) acc = fma2(h[1], c[1], acc);
        const float2 v = split(acc);
        return v.x + v.y;
      }
    };
    auto save = [&](int t) {           // the state before token t
      if (MODE == kSsmOut && P.states[r] != nullptr && t % kSsmRun == 0) {
        const int64_t run = (tok0 + t) / kSsmRun, runs = (P.s + kSsmRun - 1) / kSsmRun;
        store_states(P.states[r] + (at.batch * runs + run) * state_step + state_at, h);
      }
    };
    SsmMarks marks{0u, 0};
    if (packed && (kBack || tok0 + n_tok > known)) {
      marks = ssm_marks(P, tok0, n_tok);
      const int last = __shfl_sync(kAll, marks.seq, n_tok - 1);
      known = last + 1 < P.n_seqs ? __ldg(P.cu_seqlens + last + 1) : P.s;
    }
    if (marks.starts == 0u && n_tok == T) {
      // a saved state's run at a time, its sums kept in registers: without a store in
      // between, a run's loads and exponentials go ahead of its states
#pragma unroll 1
      for (int r0 = 0; r0 < T; r0 += kSsmRun) {
        save(r0);
        float kept[kSsmRun / G];
#pragma unroll
        for (int g0 = 0; g0 < kSsmRun; g0 += G) {
          float part[G];
#pragma unroll
          for (int g = 0; g < G; ++g) part[g] = token(kBack ? T - 1 - r0 - g0 - g : r0 + g0 + g);
          if constexpr (MODE == kSsmOut) {
            sum_over<G, G>(part, lane, 1);
            kept[g0 / G] = part[0];
          }
        }
        if constexpr (MODE == kSsmOut) {
#pragma unroll
          for (int g0 = 0; g0 < kSsmRun; g0 += G)
            *reinterpret_cast<float*>(ybuf + (r0 + g0 + lane % G) * W::kYRow + (lane / G) * 4) =
                kept[g0 / G];
        }
      }
    } else {
      for (int i = 0; i < n_tok; ++i) {
        const int t = kBack ? n_tok - 1 - i : i;
        save(t);
        const bool start = (marks.starts >> t) & 1u;
        const int seq = __shfl_sync(kAll, marks.seq, t);
        if (!kBack && start) {
          if (MODE == kSsmOut && cur >= 0 && P.hT[r] != nullptr)
            store_states(P.hT[r] + cur * state_step + state_at, h);
          cur = seq;
          load_states_or_zero(P.h0[r], cur * state_step + state_at, h);
        }
        float part[1] = {token(t)};
        if constexpr (MODE == kSsmOut) {
          sum_over<1, G>(part, lane, 1);
          if (lane % G == 0)
            *reinterpret_cast<float*>(ybuf + t * W::kYRow + (lane / G) * 4) = part[0];
        }
        if (kBack && start && tok0 + t > 0) {
          cur = find_seq(P.cu_seqlens, P.n_seqs, tok0 + t - 1);
          load_states_or_zero(P.dhT[r], cur * state_step + state_at, h);
        }
      }
    }
    sum += steps;

    // a lane's token: the outputs of the warp's channels
    if constexpr (MODE == kSsmOut) {
      __syncwarp();
      Pack<DT, CW> p;
      F2 u[CW / 2], y[CW / 2];
      lds_pack(p, st + (T + lane) * W::kRow);
      unpack_pairs(p, u);
#pragma unroll
      for (int i = 0; i < CW / 2; ++i) {
        const float2 v = *reinterpret_cast<const float2*>(ybuf + lane * W::kYRow + 8 * i);
        const float2 d = *reinterpret_cast<const float2*>(param + W::kBlockCh + warp * CW + 2 * i);
        y[i] = fma2(f2(d.x, d.y), u[i], f2(v.x, v.y));
      }
      if (gated) {
        F2 z[CW / 2];
        lds_pack(p, st + (2 * T + lane) * W::kRow);
        unpack_pairs(p, z);
#pragma unroll
        for (int i = 0; i < CW / 2; ++i)
          y[i] = mul2(y[i], mul2(z[i], rcp2(add2(exp2_of<DT, false, -1>(z[i]), f2(1.f, 1.f)))));
      }
      pack_pairs(p, y);
      if (lane < n_tok)
        store_pack(P.y[r] + (at.batch * P.s + tok0 + lane) * P.ld_y + (at.ch0 + warp * CW) * E, p);
    }
  }
  if (!active) return;
  if constexpr (MODE == kSsmOut) {
    if (at.tok0 + at.len == P.s && P.hT[r] != nullptr) {
      const int64_t seq = packed ? cur : at.batch;
      if (seq >= 0) store_states(P.hT[r] + seq * state_step + state_at, h);
    }
  } else {
    store_states(P.carry + carry_at, h);
    if (lane % G == 0)
      P.steps[(at.batch * P.chunks + at.chunk) * P.t * P.c + rc + at.ch0 + ch] = sum;
  }
}

// The state that enters each chunk of a batch row, in the place of the chunk's own
// last one (BACK: the gradient that enters from behind, in the place of what it hands
// on): a thread takes one state of a channel through the chunks.
template <bool BACK>
__global__ void __launch_bounds__(256) ssm_join_kernel(const SsmParams P) {
  pdl_wait();
  const int64_t width = static_cast<int64_t>(P.t) * P.c * P.n;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= width * P.b) return;
  const int64_t batch = id / width, i = id - batch * width;
  const int64_t chan = i / P.n;
  const int r = static_cast<int>(chan / P.c);
  const int64_t own = i - static_cast<int64_t>(r) * P.c * P.n;   // of a rank's [c][n]
  const int64_t state_step = static_cast<int64_t>(P.c) * P.n;
  const bool packed = P.cu_seqlens != nullptr;
  const float a2 = P.A[i] * kLog2e;
  const float* base = BACK ? P.dhT[r] : P.h0[r];
  float x = 0.f;
  if (base != nullptr) {
    if (!packed) x = base[batch * state_step + own];
    else if (BACK) x = base[find_seq(P.cu_seqlens, P.n_seqs, P.s - 1) * state_step + own];
  }
  float* carry = P.carry + batch * P.chunks * width + i;
  const float* steps = P.steps + batch * P.chunks * P.t * P.c + chan;
  for (int n = 0; n < P.chunks; ++n) {
    const int64_t k = BACK ? P.chunks - 1 - n : n;
    bool cut = false;                  // a sequence begins in the chunk
    if (packed) {
      const int64_t end = (k + 1) * P.chunk_len < P.s ? (k + 1) * P.chunk_len : P.s;
      cut = k == 0 || find_seq(P.cu_seqlens, P.n_seqs, end - 1) !=
                          find_seq(P.cu_seqlens, P.n_seqs, k * P.chunk_len - 1);
    }
    const float handed = carry[k * width];
    carry[k * width] = x;
    float f = a2 * steps[k * P.t * P.c];
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(f));
    x = cut ? handed : fmaf(f, x, handed);
  }
}

template <int DT, int N, int MODE>
static cudaError_t launch_walk(const SsmParams& p, cudaStream_t st) {
  using W = SsmWalk<DT, N>;
  const void* fn = reinterpret_cast<const void*>(&ssm_walk_kernel<DT, N, MODE>);
  const cudaError_t e = ensure_smem_attr(fn, W::kSmem);
  if (e != cudaSuccess) return e;
  SsmParams q = p;
  q.slabs = (p.c / p.groups + W::kBlockCh - 1) / W::kBlockCh;
  void* args[] = {&q};
  const int64_t grid = static_cast<int64_t>(q.b) * q.chunks * q.t * q.groups * q.slabs;
  return launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(W::kThreads), W::kSmem, args, st);
}

template <bool BACK>
static cudaError_t launch_join(const SsmParams& p, cudaStream_t st) {
  void* args[] = {const_cast<SsmParams*>(&p)};
  const int64_t threads = static_cast<int64_t>(p.t) * p.c * p.n * p.b;
  return launch_pdl(reinterpret_cast<const void*>(&ssm_join_kernel<BACK>),
                    dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, args, st);
}

}  // namespace spb
