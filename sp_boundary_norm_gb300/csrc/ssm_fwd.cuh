// Selective scan: a block's walk along its tokens, forward and, for the gradients'
// carries, backward.
//
// A block takes 64 channels of one rank's group (32 and 16 of 32 and 64 states) and
// walks its chunk of a batch row, 16 tokens a step.  Four warps hold the states and do
// nothing else; eight ask for rows ahead (16-byte asynchronous copies) and prepare the
// next step's tokens (softplus, d u, B and C as float32); four add a channel's lanes'
// parts of the last step's sums and finish it (D u, silu(z), the stores).  All meet once
// a step.
//
// What bounds it is the chain of a token's work in the one warp of states that each of an
// SM's schedulers has: loads from shared memory, an exponential and two products a state,
// 132 clocks a token, in which the scheduler issues 74 instructions of all of its warps
// (states saved).  Of a busy SM's time its schedulers issue in 56 %, shared memory moves in
// 63 % (without the loads of B and C at all the walk took 2 % less), the exponentials take
// 32 %.  Measured on a GB300, bf16, 8 x 8192 x 1024 packed tokens of 16 states, gated: 522 us
// (556 MB; the products alone 118 us).  Without what settle2 needs it was 468, and then one
// role for all warps took 675 us, four preparing warps 472, 32 tokens a step 612, storing the
// sums every eight tokens 509; rows asked for further ahead changed nothing.
//
// A call with few blocks is cut into chunks in time: each chunk's last state
// from a zero one and the sum of its steps (a walk of 75 clocks a token), the states that
// enter each chunk (ssm_join_kernel), and then all chunks at once.
#include <type_traits>

#include "ssm.cuh"

namespace spb {

// What a walk is for.
constexpr int kSsmOut = 0;     // y, and the states
constexpr int kSsmEnds = 1;    // a chunk's last state from a zero one, the sum of its steps
constexpr int kSsmBack = 2;    // a chunk's gradient for the state before it, from a zero
                               // one, and the sum of its steps

constexpr int kSsmPart = 128;          // threads that hold states, and that finish
constexpr int kSsmPrep = 256;          // that prepare
__host__ __device__ constexpr int walk_threads(int mode) {
  return kSsmPart + kSsmPrep + (mode == kSsmOut ? kSsmPart : 0);
}
// Registers of a thread for outputs: 16 tokens' sums and decays wait in those that hold
// states (at 128 for all of them they spill, and 522 us become 666; at 176 and 112 565, at
// 224 and 96 534).  The block starts with 128 each, which is what both shares add up to.
constexpr int kSsmStateRegisters = 200, kSsmHelpRegisters = 104, kSsmRegisters = 128;
static_assert(kSsmPart * kSsmStateRegisters + (kSsmPrep + kSsmPart) * kSsmHelpRegisters ==
                  walk_threads(kSsmOut) * kSsmRegisters, "what a block has");

// Rows in shared memory are padded so that the lanes of an access use different banks.
template <int DT, int N>
struct SsmWalk {
  using L = SsmLanes<N>;
  static constexpr int E = ElemSize<DT>::value;
  static constexpr int T = kSsmTile;
  static constexpr int kBlockCh = kSsmPart / 32 * L::kChannels;
  // channels of a token that a thread prepares, and finishes
  static constexpr int V = kBlockCh * T / kSsmPrep > 2 ? kBlockCh * T / kSsmPrep : 2;
  static constexpr int VF = kBlockCh * T / kSsmPart;
  static constexpr int kStages = 5;
  static constexpr int kRow = kBlockCh * E + 16;
  static constexpr int kShared = 2 * N * E;                    // B and C of a token
  static constexpr int kStage = T * (3 * kRow + kShared);
  static constexpr int kBC = T * 2 * N * 4;                    // float32 B and C
  static constexpr int kDPart = V * 8 + (V > 2 ? 16 : 0);      // (d, d u) of V channels
  static constexpr int kDRow = kBlockCh / V * kDPart;
  static constexpr int kYRow = kBlockCh * 4 + 32;
  static constexpr int kY = T * L::kLanes * kYRow;             // of each lane of a channel
  static constexpr size_t kSmem = kStages * kStage + 2 * (kBC + T * kDRow + kY);
};

// CUTS: packed sequences that begin from zeros (and whose last states nobody wants): four
// ranks' 3984 x 1280 tokens of 52 of them 258 us, token by token where one begins 302.
template <int DT, int N, int MODE, bool CUTS>
__global__ void __launch_bounds__(walk_threads(MODE), 1)
ssm_walk_kernel(const SsmParams P) {
  using W = SsmWalk<DT, N>;
  using L = SsmLanes<N>;
  constexpr int E = W::E, S = L::kStates, K = L::kPairs, CW = L::kChannels, G = L::kLanes;
  constexpr int T = W::T, V = W::V, VF = W::VF;
  constexpr bool kBack = MODE == kSsmBack;
  extern __shared__ __align__(16) char smem[];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!kBack && blockIdx.x == 0 && warp == 0)
    check_cu_seqlens(P.cu_seqlens, P.n_seqs, P.s, P.status);
  const SsmPlace<W::kBlockCh> at(P);
  const int r = at.r;
  const int64_t rc = static_cast<int64_t>(r) * P.c;            // the rank's first channel
  char* bcs = smem + W::kStages * W::kStage;
  char* dds = bcs + 2 * W::kBC;
  char* ys = dds + 2 * T * W::kDRow;
  const int64_t row0 = at.batch * P.s + at.tok0;
  const int n_tiles = static_cast<int>((at.len + T - 1) / T);
  // step k's first token, in the order of the walk; its tokens
  auto tile_of = [&](int k) { return static_cast<int64_t>(kBack ? n_tiles - 1 - k : k) * T; };
  auto tokens_of = [&](int64_t t0) { return at.len - t0 < T ? static_cast<int>(at.len - t0) : T; };

  if (warp >= kSsmPart / 32) {
    // ------------------------------------------------------------ preparing --
    if constexpr (MODE == kSsmOut)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSsmHelpRegisters));
    const bool finisher = warp >= (kSsmPart + kSsmPrep) / 32;
    const int ht = tid - kSsmPart - (finisher ? kSsmPrep : 0);
    const bool gated = MODE != kSsmEnds && P.gated;
    // The rows that a walk reads: dt, u (back: dy), z (not for ends); B (back: C), and C.
    // A thread's pieces of 16 bytes lie `kRows` (`kRowsB`) tokens apart.
    constexpr int kPieces = W::kBlockCh * E / 16, kRows = kSsmPrep / kPieces;
    constexpr int kPiecesB = N * E / 16, kRowsB = kSsmPrep / kPiecesB;
    static_assert(kSsmPrep % kPieces == 0 && kSsmPrep % kPiecesB == 0, "whole rows");
    const int tok_p = ht / kPieces, at_p = ht % kPieces * 16;
    const int tok_b = ht / kPiecesB, at_b = ht % kPiecesB * 16;
    const bool live_p = at_p < at.live * E;
    const int64_t lds[3] = {P.ld_dt, kBack ? P.ld_dy : P.ld_u, P.ld_z};
    const int64_t ld_b = kBack ? P.ld_C : P.ld_B;
    const int64_t row_p = row0 + tile_of(0) + tok_p, row_b = row0 + tile_of(0) + tok_b;
    const char* src[3] = {P.dt[r] + row_p * P.ld_dt + at.ch0 * E + at_p,
                          (kBack ? P.dy[r] : P.u[r]) + row_p * lds[1] + at.ch0 * E + at_p,
                          gated ? P.z[r] + row_p * P.ld_z + at.ch0 * E + at_p : nullptr};
    const char* src_b = (kBack ? P.C[r] : P.B[r]) + row_b * ld_b + at.group * N * E + at_b;
    const char* src_c = P.C[r] + row_b * P.ld_C + at.group * N * E + at_b;
    char* put = smem;                  // the stage of the next step asked for
    int asked = 0;
    auto ask = [&] {                   // the rows of the next step that is not yet asked for
      if (asked < n_tiles) {
        const int n_tok = tokens_of(tile_of(asked));
        char* dst = put + tok_p * W::kRow + at_p;
#pragma unroll
        for (int i = 0; i * kRows < T; ++i) {
          if (live_p && tok_p + i * kRows < n_tok && tok_p + i * kRows < T) {
            cp_async16(dst + i * kRows * W::kRow, src[0] + i * kRows * lds[0]);
            cp_async16(dst + (T + i * kRows) * W::kRow, src[1] + i * kRows * lds[1]);
            if (gated) cp_async16(dst + (2 * T + i * kRows) * W::kRow, src[2] + i * kRows * lds[2]);
          }
        }
        char* sh = put + 3 * T * W::kRow + tok_b * W::kShared + at_b;
#pragma unroll
        for (int i = 0; i * kRowsB < T; ++i) {
          if (tok_b + i * kRowsB < n_tok && tok_b + i * kRowsB < T) {
            cp_async16(sh + i * kRowsB * W::kShared, src_b + i * kRowsB * ld_b);
            if (MODE == kSsmOut)
              cp_async16(sh + i * kRowsB * W::kShared + N * E, src_c + i * kRowsB * P.ld_C);
          }
        }
        constexpr int kStep = kBack ? -T : T;
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (i < 2 || gated) src[i] += kStep * lds[i];
        src_b += kStep * ld_b;
        src_c += kStep * P.ld_C;
        put = put == smem + (W::kStages - 1) * W::kStage ? smem : put + W::kStage;
        ++asked;
      }
      cp_async_commit();
    };
    // v times silu(z) of VG channels, which lie at `z`
    auto gate = [&](const char* at_z, auto& v) {
      constexpr int VG = 2 * sizeof(v) / sizeof(F2);
      Pack<DT, VG> p;
      F2 z[VG / 2];
      lds_pack(p, at_z);
      unpack_pairs(p, z);
#pragma unroll
      for (int i = 0; i < VG / 2; ++i)
        v[i] = mul2(v[i], mul2(z[i], rcp2(add2(exp2_of<DT, false, -1>(z[i]), f2(1.f, 1.f)))));
    };
    // two of the block's channels' parameters (0 where there are none)
    auto param = [&](const float* from, int c) {
      return from != nullptr && c < at.live ? *reinterpret_cast<const F2*>(from + rc + at.ch0 + c)
                                            : F2(0);
    };
    const char* st = smem;             // the stage of the step being prepared, or finished
    auto next_stage = [&] {
      st = st == smem + (W::kStages - 1) * W::kStage ? smem : st + W::kStage;
    };
    if (finisher) {
      const int my = ht / (W::kBlockCh / VF), ch = ht % (W::kBlockCh / VF) * VF;
      F2 skip[VF / 2];
#pragma unroll
      for (int i = 0; i < VF / 2; ++i) skip[i] = param(P.D, ch + 2 * i);
      char* y = MODE == kSsmOut ? P.y[r] + (row0 + my) * P.ld_y + (at.ch0 + ch) * E : nullptr;
      for (int k = -1; k < n_tiles + 1; ++k) {
        meet<walk_threads(MODE)>();
        if (k < 1) continue;
        if (ch < at.live && my < tokens_of(tile_of(k - 1))) {
          const char* from = ys + ((k - 1) & 1) * W::kY + my * G * W::kYRow + ch * 4;
          Pack<DT, VF> p;
          F2 u[VF / 2], v[VF / 2];
          lds_pack(p, st + (T + my) * W::kRow + ch * E);
          unpack_pairs(p, u);
#pragma unroll
          for (int i = 0; i < VF / 2; ++i) {
            v[i] = mul2(skip[i], u[i]);
#pragma unroll
            for (int g = 0; g < G; ++g)
              v[i] = add2(v[i], *reinterpret_cast<const F2*>(from + g * W::kYRow + 8 * i));
          }
          if (gated) gate(st + (2 * T + my) * W::kRow + ch * E, v);
          pack_pairs(p, v);
          store_pack(y, p);
        }
        y += T * P.ld_y;
        next_stage();
      }
      return;
    }
    const int my = ht / (W::kBlockCh / V), part = ht % (W::kBlockCh / V);
    F2 bias[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) bias[i] = param(P.dt_bias, part * V + 2 * i);
    auto prepare = [&](int k) {
      if (my < T) {
        Pack<DT, V> p;
        F2 d[V / 2], v[V / 2];
        lds_pack(p, st + my * W::kRow + part * V * E);
        unpack_pairs(p, d);
        lds_pack(p, st + (T + my) * W::kRow + part * V * E);
        unpack_pairs(p, v);
        if (kBack && gated) gate(st + (2 * T + my) * W::kRow + part * V * E, v);
        char* dst = dds + (k & 1) * T * W::kDRow + my * W::kDRow + part * W::kDPart;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          d[i] = add2(d[i], bias[i]);
          if (P.softplus) d[i] = softplus2<DT>(d[i], nullptr);
          if constexpr (!kBack) v[i] = mul2(d[i], v[i]);
          const float2 a = split(d[i]), b = split(v[i]);
          *reinterpret_cast<float4*>(dst + 16 * i) = make_float4(a.x, a.y, b.x, b.y);
        }
      }
      const char* sh = st + 3 * T * W::kRow;
      float* bc = reinterpret_cast<float*>(bcs + (k & 1) * W::kBC);
#pragma unroll
      for (int i = ht; i < T * 2 * N / 4; i += kSsmPrep) {
        if (MODE != kSsmOut && (i * 4) % (2 * N) >= N) continue;
        Pack<DT, 4> q;
        float f[4];
        lds_pack(q, sh + i * 4 * E);
        unpack(q, f);
        *reinterpret_cast<float4*>(bc + i * 4) = make_float4(f[0], f[1], f[2], f[3]);
      }
    };
    ask();
    ask();
    for (int k = -1; k < n_tiles + (MODE == kSsmOut ? 1 : 0); ++k) {
      cp_async_wait<1>();              // step k + 1's rows
      meet<walk_threads(MODE)>();
      ask();
      if (k + 1 >= n_tiles) continue;
      prepare(k + 1);
      next_stage();
    }
    return;
  }

  // ---------------------------------------------------------------- states --
  if constexpr (MODE == kSsmOut)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSsmStateRegisters));
  const bool active = warp * CW + lane / G * 2 < at.live;      // of a lane: its two channels
  const int n0 = (lane % G) * S, ch = active ? warp * CW + lane / G * 2 : 0;
  // this lane's states: of [t * c][n], and of a rank's [sequences][c][n]; of its second
  // channel N further
  const int64_t mine = (rc + at.ch0 + ch) * N + n0;
  const int64_t state_at = static_cast<int64_t>(at.ch0 + ch) * N + n0;
  const int64_t state_step = static_cast<int64_t>(P.c) * N;
  const int64_t carry_at = (at.batch * P.chunks + at.chunk) * P.t * P.c * N + mine;
  const bool packed = P.cu_seqlens != nullptr;
  F2 h[2][K];
  float a2[2][S];
  auto load_both = [&](const float* base, int64_t i, F2 (&x)[2][K]) {
    load_states_or_zero(base, i, x[0]);
    load_states_or_zero(base, i + N, x[1]);
  };
  auto store_both = [&](float* base, int64_t i, const F2 (&x)[2][K]) {
    if (!active) return;
    store_states(base + i, x[0]);
    store_states(base + i + N, x[1]);
  };
  load_both(P.A, mine, h);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int p = 0; p < K; ++p) {
      const float2 v = split(mul2(h[c][p], f2(kLog2e, kLog2e)));
      a2[c][2 * p] = v.x;
      a2[c][2 * p + 1] = v.y;
    }
  int cur = -1;                        // the packed sequence that the state belongs to
  int64_t known = 0;                   // packed: no sequence begins in [tile, known)
  clear(h[0]);
  clear(h[1]);
  if constexpr (MODE == kSsmOut) {
    if (P.chunks > 1) load_both(P.carry, carry_at, h);
    else if (!packed) load_both(P.h0[r], at.batch * state_step + state_at, h);
  }
  if (packed && at.tok0 > 0) cur = find_seq(P.cu_seqlens, P.n_seqs, at.tok0 - 1);
  if (packed && MODE == kSsmOut && at.chunk == 0 && P.hT[r] != nullptr && P.hT[r] != P.h0[r]) {
    // the states of sequences without a token pass
    for (int j = 0; j < P.n_seqs; ++j) {
      if (__ldg(P.cu_seqlens + j) != __ldg(P.cu_seqlens + j + 1)) continue;
      F2 v[2][K];
      load_both(P.h0[r], j * state_step + state_at, v);
      store_both(P.hT[r], j * state_step + state_at, v);
    }
  }
  F2 sum = 0;                          // of the chunk's steps
  const int dd_at = ch / V * W::kDPart + ch % V * 8;
  const int64_t runs = (P.s + kSsmRun - 1) / kSsmRun;

  meet<walk_threads(MODE)>();                // (the preparers' step -1)
  for (int k = 0; k < n_tiles; ++k) {
    meet<walk_threads(MODE)>();
    const float* shared = reinterpret_cast<const float*>(bcs + (k & 1) * W::kBC) + n0;
    const char* dd = dds + (k & 1) * T * W::kDRow + dd_at;
    char* ybuf = ys + (k & 1) * W::kY + (lane % G) * W::kYRow + (warp * CW + lane / G * 2) * 4;
    const int64_t t0 = tile_of(k), tok0 = at.tok0 + t0;
    const int n_tok = tokens_of(t0);
    F2 steps = 0;
    F2 all[2][K];                      // the product of the step's decays (settle2)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int p = 0; p < K; ++p) all[c][p] = f2(1.f, 1.f);
    // one token: the states after it, and this lane's parts of its channels' sums with C;
    // ALONE: with a decay of its own
    auto token = [&](int t, auto alone) -> float2 {
      constexpr bool ALONE = decltype(alone)::value;
      const float4 v = *reinterpret_cast<const float4*>(dd + t * W::kDRow);
      const float d[2] = {v.x, v.y}, in[2] = {v.z, v.w};
      steps = add2(steps, f2(v.x, v.y));
      F2 b[K];
      load_states(shared + t * 2 * N, b);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int p = 0; p < K; ++p) {
          const F2 x = mul2(f2(d[c], d[c]), f2(a2[c][2 * p], a2[c][2 * p + 1]));
          const F2 a = ALONE ? decay2(x) : pow2(x);
          if constexpr (!ALONE) all[c][p] = mul2(all[c][p], a);
          if constexpr (kBack) {
            h[c][p] = mul2(a, fma2(f2(in[c], in[c]), b[p], h[c][p]));
          } else {
            h[c][p] = fma2(a, h[c][p], mul2(f2(in[c], in[c]), b[p]));
          }
        }
      }
      if constexpr (MODE == kSsmOut) {
        F2 q[K];
        load_states(shared + t * 2 * N + N, q);
        float part[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          F2 acc = mul2(h[c][0], q[0]);
          if constexpr (K == 2) acc = fma2(h[c][1], q[1], acc);
          const float2 x = split(acc);
          part[c] = x.x + x.y;
        }
        return make_float2(part[0], part[1]);
      }
      return make_float2(0.f, 0.f);
    };
    auto put = [&](int t, float2 part) {
      if constexpr (MODE == kSsmOut) *reinterpret_cast<float2*>(ybuf + t * G * W::kYRow) = part;
    };
    if (MODE == kSsmOut && P.states[r] != nullptr)
      store_both(P.states[r], (at.batch * runs + tok0 / kSsmRun) * state_step + state_at, h);
    SsmMarks marks{0u, 0};
    if (packed && (kBack || tok0 + n_tok > known)) {
      marks = ssm_marks(P, tok0, n_tok);
      const int last = __shfl_sync(kAll, marks.seq, n_tok - 1);
      known = last + 1 < P.n_seqs ? __ldg(P.cu_seqlens + last + 1) : P.s;
    }
    if (marks.starts == 0u && n_tok == T) {
      // the sums wait in registers: without a store in between, a step's loads and
      // exponentials go ahead of its states
      float2 part[T];
#pragma unroll
      for (int t = 0; t < T; ++t) part[t] = token(kBack ? T - 1 - t : t, std::false_type{});
      const float2 step = split(steps);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int p = 0; p < K; ++p)
          h[c][p] = mul2(h[c][p], settle2(mul2(c == 0 ? f2(step.x, step.x) : f2(step.y, step.y),
                                               f2(a2[c][2 * p], a2[c][2 * p + 1])), all[c][p]));
#pragma unroll
      for (int t = 0; t < T; ++t) put(t, part[t]);
    } else if (CUTS && n_tok == T) {
      // the same, and sequences begin (16 tokens' lost digits at most, once a sequence)
      float2 part[T];
      auto cut = [&](int t) {
        const bool zero = (marks.starts >> t) & 1u;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int p = 0; p < K; ++p) h[c][p] = zero ? F2(0) : h[c][p];
      };
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const int t = kBack ? T - 1 - i : i;
        if constexpr (!kBack) cut(t);
        part[i] = token(t, std::false_type{});
        if constexpr (kBack) cut(t);
      }
#pragma unroll
      for (int i = 0; i < T; ++i) put(kBack ? T - 1 - i : i, part[i]);
    } else {
#pragma unroll 1
      for (int i = 0; i < n_tok; ++i) {
        const int t = kBack ? n_tok - 1 - i : i;
        const bool start = (marks.starts >> t) & 1u;
        const int seq = __shfl_sync(kAll, marks.seq, t);
        if (!kBack && start) {
          if (MODE == kSsmOut && cur >= 0 && P.hT[r] != nullptr)
            store_both(P.hT[r], cur * state_step + state_at, h);
          cur = seq;
          load_both(P.h0[r], cur * state_step + state_at, h);
        }
        put(t, token(t, std::true_type{}));
        if (kBack && start && tok0 + t > 0) {
          cur = find_seq(P.cu_seqlens, P.n_seqs, tok0 + t - 1);
          load_both(P.dhT[r], cur * state_step + state_at, h);
        }
      }
    }
    sum = add2(sum, steps);
  }
  if constexpr (MODE == kSsmOut) {
    meet<walk_threads(MODE)>();              // (the preparers finish the last step)
    if (at.tok0 + at.len == P.s && P.hT[r] != nullptr) {
      const int64_t seq = packed ? cur : at.batch;
      if (seq >= 0) store_both(P.hT[r], seq * state_step + state_at, h);
    }
  } else {
    store_both(P.carry, carry_at, h);
    if (active && lane % G == 0)
      *reinterpret_cast<F2*>(P.steps + (at.batch * P.chunks + at.chunk) * P.t * P.c + rc +
                                 at.ch0 + ch) = sum;
  }
}

// Chunks whose values are asked for before the first is used (32: no faster).
constexpr int kJoinAhead = 8;

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
  constexpr int kAhead = kJoinAhead;
  for (int n0 = 0; n0 < P.chunks; n0 += kAhead) {
    float handed[kAhead], passed[kAhead];
    bool cut[kAhead];                  // a sequence begins in the chunk
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (n0 + i >= P.chunks) break;
      const int64_t k = BACK ? P.chunks - 1 - n0 - i : n0 + i;
      handed[i] = carry[k * width];
      passed[i] = steps[k * P.t * P.c];
      cut[i] = false;
      if (packed) {
        const int64_t end = (k + 1) * P.chunk_len < P.s ? (k + 1) * P.chunk_len : P.s;
        cut[i] = k == 0 || find_seq(P.cu_seqlens, P.n_seqs, end - 1) !=
                               find_seq(P.cu_seqlens, P.n_seqs, k * P.chunk_len - 1);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (n0 + i >= P.chunks) break;
      const int64_t k = BACK ? P.chunks - 1 - n0 - i : n0 + i;
      carry[k * width] = x;
      // (A > 0: a chunk's decay may overflow where the state behind it is zero or small)
      const float half = decay(0.5f * a2 * passed[i]);
      x = cut[i] || x == 0.f ? handed[i] : fmaf(half, half * x, handed[i]);
    }
  }
}

// Registers that a thread of the kernel starts with (0: unknown).
template <typename F>
static int registers_of(F* fn) {
  cudaFuncAttributes a{};
  return cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(fn)) == cudaSuccess ? a.numRegs : 0;
}

template <int DT, int N, int MODE>
static cudaError_t launch_walk(const SsmParams& p, cudaStream_t st) {
  using W = SsmWalk<DT, N>;
  const bool cuts = p.cu_seqlens != nullptr &&
                    (MODE == kSsmBack ? p.dhT[0] == nullptr
                                      : p.h0[0] == nullptr && (MODE != kSsmOut || p.hT[0] == nullptr));
  const void* fn = cuts ? reinterpret_cast<const void*>(&ssm_walk_kernel<DT, N, MODE, true>)
                        : reinterpret_cast<const void*>(&ssm_walk_kernel<DT, N, MODE, false>);
  const cudaError_t e = ensure_smem_attr(fn, W::kSmem);
  if (e != cudaSuccess) return e;
  if constexpr (MODE == kSsmOut) {
    // (with fewer to start with, the threads that hold states would wait for ever)
    static const int registers[2] = {registers_of(&ssm_walk_kernel<DT, N, MODE, false>),
                                     registers_of(&ssm_walk_kernel<DT, N, MODE, true>)};
    if (registers[cuts] < kSsmRegisters) return cudaErrorLaunchOutOfResources;
  }
  SsmParams q = p;
  q.slabs = (p.c / p.groups + W::kBlockCh - 1) / W::kBlockCh;
  void* args[] = {&q};
  const int64_t grid = static_cast<int64_t>(q.b) * q.chunks * q.t * q.groups * q.slabs;
  return launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(walk_threads(MODE)), W::kSmem, args, st);
}

template <bool BACK>
static cudaError_t launch_join(const SsmParams& p, cudaStream_t st) {
  void* args[] = {const_cast<SsmParams*>(&p)};
  const int64_t threads = static_cast<int64_t>(p.t) * p.c * p.n * p.b;
  return launch_pdl(reinterpret_cast<const void*>(&ssm_join_kernel<BACK>),
                    dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, args, st);
}

}  // namespace spb
