// Selective scan, backward.  With e = dy silu(z), along the tokens from the last:
//   G[i] = C[i] e[i] + a[i+1] G[i+1],   a = exp(d A)
//   dC[i] = sum over a group's channels of e h,  dB[i] = the same of G d u
//   g = a G h[i-1],   d(d u) = sum_n G B,   d(d) = sum_n g A + u d(d u)
//   dA = sum over tokens of g d
// A block takes its channels' chunk from the end, eight tokens a step, with warps that
// hold states and warps that prepare and finish as in the forward's walk.  Two steps are
// a run of 16 tokens: the warps that hold states start from the one that the forward
// saved for it, the upper step first.  They go through a step's tokens once forwards,
// keeping the states in registers, and once backwards, computing the decays again (16
// tokens' states do not fit, so the lower step's are computed twice).  A channel's sums
// over its states are added up by the finishing warps from its lanes' parts.  dB and dC of a token are
// summed over a lane's two channels, a warp's lanes, the block's warps, and by a second
// kernel over the blocks of a group's channels: always in the same order.
//
// The sums over a warp's lanes need no selections: the lanes' states are in an order of
// their own, state (j xor m) in place j for the lane m of a channel's, so that a lane
// keeps its even places and hands on its odd ones whichever it is; B and C lie in shared
// memory in each of these orders.
//
// What bounds it is, as in the forward's walk, one warp of states a scheduler: 447 clocks a
// token, in which the scheduler issues 199 instructions of its two warps (in 46 % of the
// time; shared memory moves in 45 %).  Measured on a GB300, bf16, 8 x 8192 x 1024 tokens of 16
// states, gated: 1768 us, 1646 without what settle2 needs.  Its inputs and outputs, 944 MB,
// the saved states, 268, and its parts of dB and dC, 134, would take 200, its products 430.
// Not faster: decays kept in
// registers (the same), two states a lane in twice the warps (a quarter slower: d, B, C
// and the parts go through shared memory twice as often), the next step's way there beside
// this one's way back (a quarter slower), eight helping warps or registers handed between
// the roles (both spill).
#include <type_traits>

#include "ssm_fwd.cuh"

namespace spb {

// Sums over tokens are taken up by second ones every so many steps: 8192 terms added one
// by one lost a quarter more of dA's digits than the rest of the arithmetic does.
constexpr int kSumSteps = 32;
// Kinds of runs.
constexpr int kBackWhole = 0, kBackCut = 1, kBackSlow = 2;
constexpr int kBackHelp = 128;         // threads that prepare and finish
constexpr int kBackThreads = kSsmPart + kBackHelp;

template <int DT, int N>
struct SsmBack {
  using L = SsmLanes<N>;
  static constexpr int E = ElemSize<DT>::value;
  static constexpr int H = kSsmRun / 2;                        // tokens of a step
  static constexpr int kWarps = kSsmPart / 32;                 // that hold states
  static constexpr int kBlockCh = kWarps * L::kChannels;
  static constexpr int kAbreast = 32 / L::kLanes;              // lanes of a warp with the same states
  static constexpr int V = kBlockCh * H / kBackHelp > 2 ? kBlockCh * H / kBackHelp : 2;   // channels that
                                                               // a thread prepares of a token
  static constexpr int kOrders = kAbreast < L::kStates ? kAbreast : L::kStates;
  static constexpr int kRow = kBlockCh * E + 16;
  static constexpr int kShared = 2 * N * E;
  static constexpr int kStage = H * (4 * kRow + kShared);      // dt, u, dy, z; B and C
  static constexpr int kBC = H * kOrders * 2 * N * 4;          // B, then C, in every order
  static constexpr int kDRow = kBlockCh * 8;                   // (d, d u) of a channel
  static constexpr int kERow = kBlockCh * 4;
  static constexpr int kYRow = kBlockCh * 4 + 32;
  static constexpr int kY = H * L::kLanes * kYRow;             // a lane's parts of one sum
  static constexpr int kSum = H * 2 * N * 4;                   // dB and dC of a warp's step
  static constexpr int kWhole = kSsmPart * L::kStates * 2 * 4; // dA so far, a lane's
  // four steps' rows, and what is prepared of them; two steps' sums
  static constexpr size_t kSmem =
      4 * (kStage + kBC + H * (kDRow + kERow)) + 2 * (3 * kY + kWarps * kSum) + kWhole;
};

// CUTS: packed sequences that begin from zeros: four ranks' 3984 x 1280 tokens of 52 of them
// 721 us, where runs with a beginning were walked token by token 917.  (A kernel of its own:
// beside that code the other's registers spill, 8 x 8192 x 1024 both directions 2122 -> 2345.)
template <int DT, int N, bool CUTS>
__global__ void __launch_bounds__(kBackThreads, 1)
ssm_bwd_kernel(const SsmParams P) {
  using W = SsmBack<DT, N>;
  using L = SsmLanes<N>;
  constexpr int E = W::E, S = L::kStates, K = L::kPairs, CW = L::kChannels, G = L::kLanes;
  constexpr int H = W::H, T = kSsmRun, CB = W::kBlockCh, O = W::kOrders;
  extern __shared__ __align__(16) char smem[];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == 0 && warp == 0)
    check_cu_seqlens(P.cu_seqlens, P.n_seqs, P.s, P.status);
  const SsmPlace<CB> at(P);
  const int r = at.r;
  const int64_t rc = static_cast<int64_t>(r) * P.c;
  char* bcs = smem + 4 * W::kStage;
  char* dds = bcs + 4 * W::kBC;
  char* es = dds + 4 * H * W::kDRow;
  char* outs = es + 4 * H * W::kERow;                          // [2][3] of kY
  char* sums = outs + 6 * W::kY;
  const int64_t row0 = at.batch * P.s + at.tok0;
  const int n_runs = static_cast<int>((at.len + T - 1) / T), n_steps = 2 * n_runs;
  // step k's first token of the chunk, and its tokens: the upper half of a run, the lower
  auto first_of = [&](int k) {
    return static_cast<int64_t>(n_runs - 1 - (k >> 1)) * T + (k & 1 ? 0 : H);
  };
  auto tokens_of = [&](int k) {
    const int64_t left = at.len - first_of(k);
    return left < 0 ? 0 : left < H ? static_cast<int>(left) : H;
  };
  const bool gated = P.gated != 0;

  if (warp >= W::kWarps) {
    // ------------------------------------------------- preparing, finishing --
    const int ht = tid - kSsmPart;
    // pieces of 16 bytes of a step's rows, a thread's `kRows` tokens apart
    constexpr int kPieces = CB * E / 16, kRows = kBackHelp / kPieces;
    constexpr int kPiecesB = N * E / 16, kRowsB = kBackHelp / kPiecesB;
    static_assert(kBackHelp % kPieces == 0 && kBackHelp % kPiecesB == 0, "whole rows");
    const int tok_p = ht / kPieces, at_p = ht % kPieces * 16;
    const int tok_b = ht / kPiecesB, at_b = ht % kPiecesB * 16;
    const bool live_p = at_p < at.live * E;
    const char* src[4] = {P.dt[r] + at.ch0 * E + at_p, P.u[r] + at.ch0 * E + at_p,
                          P.dy[r] + at.ch0 * E + at_p, gated ? P.z[r] + at.ch0 * E + at_p : nullptr};
    const char* src_b = P.B[r] + at.group * N * E + at_b;
    const char* src_c = P.C[r] + at.group * N * E + at_b;
    auto ask = [&](int k) {
      if (k < n_steps) {
        const int n_tok = tokens_of(k);
        const int64_t row = row0 + first_of(k);
        char* st = smem + (k & 3) * W::kStage;
#pragma unroll
        for (int i = 0; i < H; i += kRows) {
          const int tok = tok_p + i;
          if (live_p && tok < n_tok) {
            char* dst = st + tok * W::kRow + at_p;
            cp_async16(dst, src[0] + (row + tok) * P.ld_dt);
            cp_async16(dst + H * W::kRow, src[1] + (row + tok) * P.ld_u);
            cp_async16(dst + 2 * H * W::kRow, src[2] + (row + tok) * P.ld_dy);
            if (gated) cp_async16(dst + 3 * H * W::kRow, src[3] + (row + tok) * P.ld_z);
          }
        }
#pragma unroll
        for (int i = 0; i < H; i += kRowsB) {
          const int tok = tok_b + i;
          if (tok < n_tok) {
            char* sh = st + 4 * H * W::kRow + tok * W::kShared + at_b;
            cp_async16(sh, src_b + (row + tok) * P.ld_B);
            cp_async16(sh + N * E, src_c + (row + tok) * P.ld_C);
          }
        }
      }
      cp_async_commit();
    };
    // a thread's channels of a token
    constexpr int V = W::V;
    const int my = ht / (CB / V), ch = ht % (CB / V) * V;
    const bool mine = my < H, live = ch < at.live;
    F2 bias[V / 2], skip[V / 2], dD[V / 2], dbias[V / 2], all_D[V / 2], all_bias[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      auto param = [&](const float* from) {
        return from != nullptr && live ? *reinterpret_cast<const F2*>(from + rc + at.ch0 + ch + 2 * i)
                                       : F2(0);
      };
      bias[i] = param(P.dt_bias);
      skip[i] = param(P.D);
      dD[i] = dbias[i] = all_D[i] = all_bias[i] = 0;
    }
    auto take_up = [&] {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        all_D[i] = add2(all_D[i], dD[i]);
        all_bias[i] = add2(all_bias[i], dbias[i]);
        dD[i] = dbias[i] = 0;
      }
    };
    // what is kept of a token's channels until its sums are there
    struct Kept {
      F2 d[V / 2], u[V / 2], e[V / 2], slope[V / 2], dz[V / 2];
    };
    auto prepare = [&](int k, Kept& x) {
      const char* st = smem + (k & 3) * W::kStage;
      if (mine) {
        const char* from = st + my * W::kRow + ch * E;
        Pack<DT, V> p;
        auto read = [&](int a, F2 (&v)[V / 2]) {
          lds_pack(p, from + a * H * W::kRow);
          unpack_pairs(p, v);
#pragma unroll
          for (int i = 0; i < V / 2; ++i) v[i] = live ? v[i] : F2(0);   // (a dead channel adds zeros)
        };
        F2 z[V / 2];
        read(0, x.d);
        read(1, x.u);
        read(2, x.e);
        if (gated) read(3, z);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          x.d[i] = add2(x.d[i], bias[i]);
          x.slope[i] = f2(1.f, 1.f);
          if (P.softplus) x.d[i] = softplus2<DT>(x.d[i], &x.slope[i]);
          if (gated) {
            // sg = sigmoid(z); silu' = sg + z sg (1 - sg)
            const F2 sg = rcp2(add2(exp2_of<DT, false, -1>(z[i]), f2(1.f, 1.f)));
            const F2 silu = mul2(z[i], sg);
            x.dz[i] = mul2(x.e[i], fma2(silu, fma2(sg, f2(-1.f, -1.f), f2(1.f, 1.f)), sg));
            x.e[i] = mul2(x.e[i], silu);
          }
          const float2 a = split(x.d[i]), b = split(mul2(x.d[i], x.u[i]));
          *reinterpret_cast<float4*>(dds + ((k & 3) * H + my) * W::kDRow + (ch + 2 * i) * 8) =
              make_float4(a.x, b.x, a.y, b.y);
          *reinterpret_cast<F2*>(es + ((k & 3) * H + my) * W::kERow + (ch + 2 * i) * 4) = x.e[i];
        }
      }
      // B and C, four (two) states at a time, in every order
      const char* sh = st + 4 * H * W::kRow;
      float* bc = reinterpret_cast<float*>(bcs + (k & 3) * W::kBC);
      constexpr int kQuads = H * 2 * N / S;
#pragma unroll
      for (int i = ht; i < kQuads * O; i += kBackHelp) {
        const int m = i % O, quad = i / O;
        const int tok = quad / (2 * N / S), e = quad % (2 * N / S) * S;
        Pack<DT, S> p;
        float f[S];
        lds_pack(p, sh + tok * W::kShared + e * E);
        unpack(p, f);
        float* to = bc + ((tok * 2 + (e >= N)) * O + m) * N + e % N;
        if (m & 1) {
#pragma unroll
          for (int j = 0; j < S; j += 2) {
            const float v = f[j];
            f[j] = f[j + 1];
            f[j + 1] = v;
          }
        }
        if constexpr (S == 4) {
          const bool far = m & 2;
          *reinterpret_cast<float4*>(to) = make_float4(far ? f[2] : f[0], far ? f[3] : f[1],
                                                       far ? f[0] : f[2], far ? f[1] : f[3]);
        } else {
          *reinterpret_cast<float2*>(to) = make_float2(f[0], f[1]);
        }
      }
    };
    const int live_warps = (at.live + CW - 1) / CW;
    auto finish = [&](int k, const Kept& x) {
      const int n_tok = tokens_of(k);
      const int64_t row = row0 + first_of(k);
      // dB and dC: the block's warps in order
      const char* from = sums + (k & 1) * W::kWarps * W::kSum;
#pragma unroll
      for (int i = ht; i < H * 2 * N / 4; i += kBackHelp) {
        const int tok = i / (N / 2), e = (i % (N / 2)) * 4;
        if (tok >= n_tok) continue;
        F2 both[2] = {0, 0};
        for (int w = 0; w < live_warps; ++w) {
          const float4 v = *reinterpret_cast<const float4*>(from + w * W::kSum + i * 16);
          both[0] = add2(both[0], f2(v.x, v.y));
          both[1] = add2(both[1], f2(v.z, v.w));
        }
        if (P.partial_bc != nullptr) {
          const int64_t rows = static_cast<int64_t>(P.b) * P.s;
          store_states(P.partial_bc + (at.slab * rows + row + tok) * 2 * N + e, both);
        } else {
          Pack<DT, 4> p;
          pack_pairs(p, both);
          const int n = e % N + at.group * N;
          if (e < N) store_pack(P.dB[r] + (row + tok) * P.ld_dB + n * E, p);
          else store_pack(P.dC[r] + (row + tok) * P.ld_dC + n * E, p);
        }
      }
      if (!live || my >= n_tok) return;
      // the channels' sums over their lanes
      const char* out = outs + (k & 1) * 3 * W::kY + my * G * W::kYRow + ch * 4;
      F2 du[V / 2], ddt[V / 2], dz[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        F2 through = 0, decay = 0, inner = 0;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const char* from = out + g * W::kYRow + 8 * i;
          through = add2(through, *reinterpret_cast<const F2*>(from));
          decay = add2(decay, *reinterpret_cast<const F2*>(from + W::kY));
          if (gated) inner = add2(inner, *reinterpret_cast<const F2*>(from + 2 * W::kY));
        }
        du[i] = fma2(x.d[i], through, mul2(skip[i], x.e[i]));
        ddt[i] = mul2(fma2(x.u[i], through, mul2(decay, f2(kLn2, kLn2))), x.slope[i]);
        if (gated) dz[i] = mul2(x.dz[i], fma2(skip[i], x.u[i], inner));
        dD[i] = fma2(x.e[i], x.u[i], dD[i]);
        dbias[i] = add2(dbias[i], ddt[i]);
      }
      const int64_t to = row + my, off = (at.ch0 + ch) * E;
      Pack<DT, V> p;
      pack_pairs(p, du);
      store_pack(P.du[r] + to * P.ld_du + off, p);
      pack_pairs(p, ddt);
      store_pack(P.ddt[r] + to * P.ld_ddt + off, p);
      if (gated) {
        pack_pairs(p, dz);
        store_pack(P.dz[r] + to * P.ld_dz + off, p);
      }
    };
    ask(0);
    ask(1);
    Kept kept[3];                      // of steps k - 1, k, k + 1: by k modulo 3
    auto step = [&](int k, Kept& x) {
      cp_async_wait<1>();              // step k + 2's rows
      meet<kBackThreads>();
      ask(k + 4);                      // (in the place of step k's, which are prepared)
      if (k >= 1) finish(k - 1, x);
      if (k % kSumSteps == 0) take_up();
      if (k + 2 < n_steps) prepare(k + 2, x);
    };
    for (int k = -2; k <= n_steps; k += 3) {
      step(k, kept[0]);
      if (k + 1 <= n_steps) step(k + 1, kept[1]);
      if (k + 2 <= n_steps) step(k + 2, kept[2]);
    }
    if (P.partial_params == nullptr) return;
    take_up();
    // the block's tokens of a channel, in the order of its threads
    float* to = P.partial_params + (at.batch * P.chunks + at.chunk) * P.t * P.c * (N + 2) +
                static_cast<int64_t>(P.t) * P.c * N;
    F2* sum = reinterpret_cast<F2*>(smem);                     // [2][H][CB / 2]
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      if (!mine) continue;
      sum[my * (CB / 2) + ch / 2 + i] = all_D[i];
      sum[(H + my) * (CB / 2) + ch / 2 + i] = all_bias[i];
    }
    asm volatile("bar.sync 2, %0;" ::"n"(kBackHelp) : "memory");
    if (ht < CB) {
      const int which = ht / (CB / 2), c = ht % (CB / 2);
      F2 a = 0;
#pragma unroll
      for (int i = 0; i < H; ++i) a = add2(a, sum[(which * H + i) * (CB / 2) + c]);
      if (2 * c < at.live)
        *reinterpret_cast<F2*>(to + static_cast<int64_t>(which) * P.t * P.c + rc + at.ch0 + 2 * c) = a;
    }
    return;
  }

  // ---------------------------------------------------------------- states --
  // the lane's two channels (dead ones go by the block's first, and add zeros), its order
  const int my_ch = warp * CW + lane / G * 2;
  const bool active = my_ch < at.live;
  const int order = lane / G & (O - 1), n0 = (lane % G) * S, ch = active ? my_ch : 0;
  const int64_t mine = (rc + at.ch0 + ch) * N + n0;
  const int64_t state_at = static_cast<int64_t>(at.ch0 + ch) * N + n0;
  const int64_t state_step = static_cast<int64_t>(P.c) * N;
  const int64_t all_runs = (P.s + T - 1) / T;
  const bool packed = P.cu_seqlens != nullptr;
  // to the lane's order, and back (the same)
  auto reorder = [&](F2 (&x)[2][K]) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int p = 0; p < K; ++p) {
        const float2 v = split(x[c][p]);
        x[c][p] = order & 1 ? f2(v.y, v.x) : x[c][p];
      }
      if constexpr (K == 2) {
        const F2 v = x[c][0];
        x[c][0] = order & 2 ? x[c][1] : v;
        x[c][1] = order & 2 ? v : x[c][1];
      }
    }
  };
  auto load_both = [&](const float* base, int64_t i, F2 (&x)[2][K]) {
    load_states_or_zero(base, i, x[0]);
    load_states_or_zero(base, i + N, x[1]);
    if (!active) {
      clear(x[0]);
      clear(x[1]);
    }
    reorder(x);
  };
  auto store_both = [&](float* base, int64_t i, const F2 (&x)[2][K]) {
    F2 y[2][K];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int p = 0; p < K; ++p) y[c][p] = x[c][p];
    reorder(y);
    if (!active) return;
    store_states(base + i, y[0]);
    store_states(base + i + N, y[1]);
  };
  // the gradient that comes from behind (times the decay in between); the decay rates
  // in powers of two, their gradients' sums; the state before the run, and the next run's
  F2 back[2][K], a2[2][K], dA[2][K], first[2][K], next[2][K];
  load_both(P.A, mine, a2);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int p = 0; p < K; ++p) {
      a2[c][p] = mul2(a2[c][p], f2(kLog2e, kLog2e));
      dA[c][p] = first[c][p] = 0;
    }
  if (P.chunks > 1) {
    load_both(P.carry, (at.batch * P.chunks + at.chunk) * P.t * P.c * N + mine, back);
  } else {
    const int64_t seq = packed ? find_seq(P.cu_seqlens, P.n_seqs, P.s - 1) : at.batch;
    load_both(P.dhT[r], seq * state_step + state_at, back);
  }
  if (packed && at.chunk == 0 && P.hT[r] != nullptr) {
    // the gradients of the states of sequences without a token pass
    for (int j = 0; j < P.n_seqs; ++j) {
      if (__ldg(P.cu_seqlens + j) != __ldg(P.cu_seqlens + j + 1)) continue;
      F2 v[2][K];
      load_both(P.dhT[r], j * state_step + state_at, v);
      store_both(P.hT[r], j * state_step + state_at, v);
    }
  }
  auto run_state = [&](int run) {      // (as it lies in memory)
    const int64_t i = (at.batch * all_runs + at.tok0 / T + n_runs - 1 - run) * state_step + state_at;
    load_states(P.states[r] + i, next[0]);
    load_states(P.states[r] + i + N, next[1]);
  };
  if (n_runs > 0) run_state(0);
  // dA so far, in shared memory (its registers would cost 2 % of the walk)
  F2* whole = reinterpret_cast<F2*>(sums + 2 * W::kWarps * W::kSum) + tid;
#pragma unroll
  for (int i = 0; i < 2 * K; ++i) whole[i * kSsmPart] = 0;
  auto take_up = [&] {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int p = 0; p < K; ++p) {
        whole[(c * K + p) * kSsmPart] = add2(whole[(c * K + p) * kSsmPart], dA[c][p]);
        dA[c][p] = 0;
      }
  };
  SsmMarks marks{0u, 0};
  int64_t known = P.s;                 // packed: where the sequence of the next run's last
                                       // token begins, or behind it

  meet<kBackThreads>();
  meet<kBackThreads>();                // (steps 0 and 1 are prepared)
  for (int k = 0; k < n_steps; ++k) {
    meet<kBackThreads>();
    const int half = k & 1 ? 0 : H;    // the step's first token in its run
    const int64_t run0 = at.tok0 + first_of(k) - half;
    const int n_tok = tokens_of(k);
    // what is prepared of a step
    auto shared_of = [&](int j) {
      return reinterpret_cast<const float*>(bcs + (j & 3) * W::kBC) + order * N + n0;
    };
    auto dd_of = [&](int j) { return dds + (j & 3) * H * W::kDRow + my_ch * 8; };
    const float* shared = shared_of(k);
    const char* dd = dd_of(k);
    const char* ee = es + (k & 3) * H * W::kERow + my_ch * 4;
    char* out = outs + (k & 1) * 3 * W::kY + (lane % G) * W::kYRow + my_ch * 4;
    float* put = reinterpret_cast<float*>(sums + ((k & 1) * W::kWarps + warp) * W::kSum);
    if (half != 0) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int p = 0; p < K; ++p) first[c][p] = active ? next[c][p] : F2(0);
      reorder(first);
      if (k + 2 < n_steps) run_state((k >> 1) + 1);
      if (packed) {
        marks.starts = 0;
        if (known >= run0) {
          marks = ssm_marks(P, run0, n_tok > 0 ? H + n_tok : tokens_of(k + 1));
          known = run0 > 0 ? __ldg(P.cu_seqlens + find_seq(P.cu_seqlens, P.n_seqs, run0 - 1)) : 0;
        }
      }
    }
    constexpr int kOrderStride = 2 * O * N;            // floats between tokens' B

    // SLOW: runs with less than 16 tokens, or where a sequence with states of its own
    // begins: token by token, with the states in local memory.  CUT: runs where one begins
    // from zeros.
    auto go = [&](auto mode) {
      constexpr bool SLOW = decltype(mode)::value == kBackSlow, CUT = decltype(mode)::value == kBackCut;
      constexpr int kUnroll = SLOW ? 1 : H;
      constexpr bool kSettled = !SLOW && !CUT;
      auto begins = [&](int t) { return (SLOW || CUT) && (marks.starts >> t & 1u); };
      auto enter = [&](int t, F2 (&h)[2][K]) {         // the state before token t
        if constexpr (SLOW) {
          if (begins(t))
            load_both(P.h0[r], __shfl_sync(kAll, marks.seq, t) * state_step + state_at, h);
        } else if constexpr (CUT) {
          const bool zero = begins(t);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int p = 0; p < K; ++p) h[c][p] = zero ? F2(0) : h[c][p];
        }
      };
      // the states after a token of a step
      auto token = [&](const char* dt, const float* bt, F2 (&h)[2][K]) {
        const float4 v = *reinterpret_cast<const float4*>(dt);
        const float d[2] = {v.x, v.z}, in[2] = {v.y, v.w};
        F2 b[K];
        load_states(bt, b);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int p = 0; p < K; ++p) {
            const F2 a = pow2(mul2(f2(d[c], d[c]), a2[c][p]));
            h[c][p] = fma2(a, h[c][p], mul2(f2(in[c], in[c]), b[p]));
          }
      };
      F2 begin[2][K];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int p = 0; p < K; ++p) begin[c][p] = first[c][p];
      if (half != 0 && n_tok > 0) {                    // through the lower step first
        const float* low = shared_of(k + 1);
        const char* low_d = dd_of(k + 1);
#pragma unroll kUnroll
        for (int i = 0; i < H; ++i) {
          enter(i, begin);
          token(low_d + i * W::kDRow, low + i * kOrderStride, begin);
        }
      }
      F2 h[H][2][K];
      {
        F2 now[2][K];
        float2 inner[H];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int p = 0; p < K; ++p) now[c][p] = begin[c][p];
#pragma unroll kUnroll
        for (int i = 0; i < H; ++i) {
          inner[i] = make_float2(0.f, 0.f);
          if (!SLOW || i < n_tok) {
            enter(half + i, now);
            token(dd + i * W::kDRow, shared + i * kOrderStride, now);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int p = 0; p < K; ++p) h[i][c][p] = now[c][p];
            // (also without a gate: a branch here would keep the tokens apart)
            F2 q[K];
            load_states(shared + i * kOrderStride + O * N, q);
            float sum[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              F2 acc = mul2(now[c][0], q[0]);
              if constexpr (K == 2) acc = fma2(now[c][1], q[1], acc);
              const float2 x = split(acc);
              sum[c] = x.x + x.y;
            }
            inner[i] = make_float2(sum[0], sum[1]);
          }
        }
        if (gated) {
#pragma unroll kUnroll
          for (int i = 0; i < H; ++i)
            *reinterpret_cast<float2*>(out + 2 * W::kY + i * G * W::kYRow) = inner[i];
        }
      }
      // Back.  The sums wait in registers, which the states give up, until the step's last:
      // without a store in between, loads go ahead of what is being summed.
      constexpr int kLevels = O == 4 ? 2 : 1;          // of lanes, that halve the states
      constexpr int kLeft = S >> kLevels;              // states of dB and of dC then
      constexpr int kBoth = W::kAbreast > O ? 1 : 2;   // dB and dC, or one of them
      F2 all[2][K];                                    // the step's decays together
      float steps[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int p = 0; p < K; ++p) all[c][p] = f2(1.f, 1.f);
      float4 wait[H];
      float wait_bc[H][kBoth * kLeft];
#pragma unroll kUnroll
      for (int i = H - 1; i >= 0; --i) {
        if (!SLOW || i < n_tok) {
          const int t = half + i;
          const float4 dv = *reinterpret_cast<const float4*>(dd + i * W::kDRow);
          const float2 ev = *reinterpret_cast<const float2*>(ee + i * W::kERow);
          const float d[2] = {dv.x, dv.z}, in[2] = {dv.y, dv.w}, e[2] = {ev.x, ev.y};
          F2 b[K], q[K], db[K], dc[K], before[2][K];
          load_states(shared + i * kOrderStride, b);
          load_states(shared + i * kOrderStride + O * N, q);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int p = 0; p < K; ++p)
              before[c][p] = i > 0 ? h[i > 0 ? i - 1 : 0][c][p] : begin[c][p];
          enter(t, before);
          float through[2], decay[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const F2 e2 = f2(e[c], e[c]), in2 = f2(in[c], in[c]), d2 = f2(d[c], d[c]);
            F2 to_u = 0, to_d = 0;
            if constexpr (kSettled) steps[c] += d[c];
#pragma unroll
            for (int p = 0; p < K; ++p) {
              const F2 gr = fma2(q[p], e2, back[c][p]);
              dc[p] = c == 0 ? mul2(h[i][c][p], e2) : fma2(h[i][c][p], e2, dc[p]);
              db[p] = c == 0 ? mul2(gr, in2) : fma2(gr, in2, db[p]);
              to_u = p == 0 ? mul2(gr, b[p]) : fma2(gr, b[p], to_u);
              const F2 x = mul2(d2, a2[c][p]), a = SLOW ? decay2(x) : pow2(x);
              if constexpr (kSettled) all[c][p] = mul2(all[c][p], a);
              back[c][p] = mul2(a, gr);
              const F2 g = mul2(back[c][p], before[c][p]);
              to_d = p == 0 ? mul2(g, a2[c][p]) : fma2(g, a2[c][p], to_d);
              dA[c][p] = fma2(g, d2, dA[c][p]);
            }
            const float2 y = split(to_u), w = split(to_d);
            through[c] = y.x + y.y;
            decay[c] = w.x + w.y;
          }
          if constexpr (CUT) enter(t, back);           // (and none comes from behind)
          if (SLOW && begins(t)) {
            const int64_t seq = __shfl_sync(kAll, marks.seq, t);
            if (P.hT[r] != nullptr) store_both(P.hT[r], seq * state_step + state_at, back);
            const float* from = run0 + t > 0 ? P.dhT[r] : nullptr;
            const int64_t prev =
                from != nullptr ? find_seq(P.cu_seqlens, P.n_seqs, run0 + t - 1) : 0;
            load_both(from, prev * state_step + state_at, back);
          }
          wait[i] = make_float4(through[0], through[1], decay[0], decay[1]);
          // dB and dC over the warp's lanes with the same states: keep the even places,
          // hand on the odd ones; then of two states; then dB or dC
          float v[2][S];
#pragma unroll
          for (int p = 0; p < K; ++p) {
            const float2 y = split(db[p]), w = split(dc[p]);
            v[0][2 * p] = y.x;
            v[0][2 * p + 1] = y.y;
            v[1][2 * p] = w.x;
            v[1][2 * p + 1] = w.y;
          }
#pragma unroll
          for (int level = 0; level < kLevels; ++level) {
            const int step = 1 << level;
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
              for (int j = 0; j < S; j += 2 * step)
                v[w][j] += __shfl_xor_sync(kAll, v[w][j + step], G * step);
          }
          if constexpr (kBoth == 1) {
            // lanes left over: one takes dB, the other dC (and others the same)
            static_assert(kLeft == 1, "one state");
            const bool up = lane & G * O;
            const float give = up ? v[0][0] : v[1][0];
            float keep = up ? v[1][0] : v[0][0];
            keep += __shfl_xor_sync(kAll, give, G * O);
#pragma unroll
            for (int m = 2 * O; m < W::kAbreast; m *= 2)
              keep += __shfl_xor_sync(kAll, keep, G * m);
            wait_bc[i][0] = keep;
          } else {
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
              for (int j = 0; j < kLeft; ++j) wait_bc[i][w * kLeft + j] = v[w][2 * j];
          }
        }
      }
      if constexpr (kSettled) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int p = 0; p < K; ++p)
            back[c][p] = mul2(back[c][p], settle2(mul2(f2(steps[c], steps[c]), a2[c][p]), all[c][p]));
      }
#pragma unroll kUnroll
      for (int i = 0; i < H; ++i) {
        if (SLOW && i >= n_tok) break;
        char* to = out + i * G * W::kYRow;
        *reinterpret_cast<float2*>(to) = make_float2(wait[i].x, wait[i].y);
        *reinterpret_cast<float2*>(to + W::kY) = make_float2(wait[i].z, wait[i].w);
        float* bc = put + i * 2 * N + n0;
        if constexpr (kBoth == 1) {
          bc[(lane & G * O ? N : 0) + order] = wait_bc[i][0];
        } else {
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int j = 0; j < kLeft; ++j) bc[w * N + (2 * j ^ order)] = wait_bc[i][w * kLeft + j];
        }
      }
    };
    if (k % kSumSteps == 0) take_up();
    if (n_tok == 0) continue;
    if (marks.starts == 0u && n_tok == H)
      go(std::integral_constant<int, kBackWhole>{});
    else if (CUTS && n_tok == H) go(std::integral_constant<int, CUTS ? kBackCut : kBackSlow>{});
    else go(std::integral_constant<int, kBackSlow>{});
  }
  meet<kBackThreads>();                // (the others finish the last step)
  if (!packed && at.chunk == 0 && P.hT[r] != nullptr)
    store_both(P.hT[r], at.batch * state_step + state_at, back);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int p = 0; p < K; ++p) dA[c][p] = add2(whole[(c * K + p) * kSsmPart], dA[c][p]);
  if (P.partial_params != nullptr)
    store_both(P.partial_params + (at.batch * P.chunks + at.chunk) * P.t * P.c * (N + 2), mine, dA);
}

// dB and dC: the blocks of a group's channels in order.
template <int DT>
__global__ void __launch_bounds__(256) ssm_bc_kernel(const SsmParams P) {
  pdl_wait();
  const int64_t rows = static_cast<int64_t>(P.b) * P.s;
  const int quads = P.n / 2;           // of four values, dB then dC, of a token and group
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t most = rows * quads * P.t * P.groups;
  if (id >= most) return;
  const int64_t rg = divide(id, rows * quads, most), i = id - rg * rows * quads;
  const int64_t row = divide(i, quads, most);
  const int e = static_cast<int>(i - row * quads) * 4;
  const float* from = P.partial_bc + rg * P.slabs * rows * 2 * P.n + i * 4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < P.slabs; ++k) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(from + k * rows * 2 * P.n));
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  const int r = static_cast<int>(rg / P.groups), group = static_cast<int>(rg - static_cast<int64_t>(r) * P.groups);
  Pack<DT, 4> p;
  const float f[4] = {a.x, a.y, a.z, a.w};
  pack(p, f);
  const int64_t n = (e % P.n + group * P.n) * ElemSize<DT>::value;
  if (e < P.n) store_pack(P.dB[r] + row * P.ld_dB + n, p);
  else store_pack(P.dC[r] + row * P.ld_dC + n, p);
}

// The parameters' gradients from the blocks of a channel.
static __global__ void __launch_bounds__(kPartThreads)
ssm_params_kernel(const float* from, int64_t channels, int n, int64_t parts, SsmParamGrads g) {
  pdl_wait();
  const int64_t all = channels * (n + 2);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
  const float a = sum_parts(from, all, parts, i);
  if (threadIdx.x >= 32 || i >= all) return;
  if (i < channels * n) {
    if (g.dA != nullptr) g.dA[i] = a;
  } else if (i < channels * (n + 1)) {
    if (g.dD != nullptr) g.dD[i - channels * n] = a;
  } else if (g.ddt_bias != nullptr) {
    g.ddt_bias[i - channels * (n + 1)] = a;
  }
}

template <int DT, int N>
static cudaError_t launch_back(const SsmParams& p, cudaStream_t st) {
  using W = SsmBack<DT, N>;
  const bool cuts = p.cu_seqlens != nullptr && p.h0[0] == nullptr && p.dhT[0] == nullptr &&
                    p.hT[0] == nullptr;
  const void* fn = cuts ? reinterpret_cast<const void*>(&ssm_bwd_kernel<DT, N, true>)
                        : reinterpret_cast<const void*>(&ssm_bwd_kernel<DT, N, false>);
  const cudaError_t e = ensure_smem_attr(fn, W::kSmem);
  if (e != cudaSuccess) return e;
  void* args[] = {const_cast<SsmParams*>(&p)};
  const int64_t grid = static_cast<int64_t>(p.b) * p.chunks * p.t * p.groups * p.slabs;
  return launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(kBackThreads), W::kSmem, args, st);
}

template <int DT, int N>
static cudaError_t launch_bwd(const SsmParams& p, const SsmParamGrads& g, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (p.chunks > 1) {
    e = launch_walk<DT, N, kSsmBack>(p, st);
    if (e == cudaSuccess) e = launch_join<true>(p, st);
    if (e != cudaSuccess) return e;
  }
  e = launch_back<DT, N>(p, st);
  if (e == cudaSuccess && p.partial_bc != nullptr) {
    void* args[] = {const_cast<SsmParams*>(&p)};
    const int64_t threads = static_cast<int64_t>(p.b) * p.s * (p.n / 2) * p.t * p.groups;
    e = launch_pdl(reinterpret_cast<const void*>(&ssm_bc_kernel<DT>),
                   dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, args, st);
  }
  if (e == cudaSuccess && p.partial_params != nullptr) {
    const float* from = p.partial_params;
    int64_t channels = static_cast<int64_t>(p.t) * p.c, parts = static_cast<int64_t>(p.b) * p.chunks;
    int n = p.n;
    SsmParamGrads grads = g;
    void* args[] = {&from, &channels, &n, &parts, &grads};
    const int64_t columns = channels * (n + 2);
    e = launch_pdl(reinterpret_cast<const void*>(&ssm_params_kernel),
                   dim3(static_cast<unsigned>((columns + 31) / 32)), dim3(kPartThreads), 0, args, st);
  }
  return e;
}

template <int DT>
cudaError_t launch_ssm_bwd_of(const SsmParams& p, const SsmParamGrads& g, cudaStream_t st) {
  switch (p.n) {
    case 8: return launch_bwd<DT, 8>(p, g, st);
    case 16: return launch_bwd<DT, 16>(p, g, st);
    case 32: return launch_bwd<DT, 32>(p, g, st);
    default: return launch_bwd<DT, 64>(p, g, st);
  }
}

}  // namespace spb
