// Selective scan, backward.  With e = dy silu(z), along the tokens from the last:
//   G[i] = C[i] e[i] + a[i+1] G[i+1],   a = exp(d A)
//   dC[i] = sum over a group's channels of e h,  dB[i] = the same of G d u
//   g = a G h[i-1],   d(d u) = sum_n G B,   d(d) = sum_n g A + u d(d u)
//   dA = sum over tokens of g d
// A block takes its channels' chunk from the end, a run of 16 tokens a step, with the
// same halves as the forward's walk.  The warps that hold states start from the one that
// the forward saved for the run: eight tokens at a time, the upper ones first, they go
// once forwards, keeping states and decays in registers, and once backwards (16 tokens
// of both do not fit, so the run's lower states are computed twice).  dB and dC of a
// token are summed over a lane's two channels, a warp's lanes, the block's warps, and
// by a second kernel over the blocks of a group's channels: always in the same order.
// The other warps keep what they have prepared of a token (u, e, the slopes of softplus
// and silu) in their registers until its sums are there.
#include <type_traits>

#include "ssm_fwd.cuh"

namespace spb {

template <int DT, int N>
struct SsmBack {
  using L = SsmLanes<N>;
  static constexpr int E = ElemSize<DT>::value;
  static constexpr int T = kSsmRun;
  static constexpr int kWarps = kSsmPart / 32;                 // that hold states
  static constexpr int kBlockCh = kWarps * L::kChannels;
  static constexpr int V = kBlockCh * T / kSsmPart;
  static constexpr int kStages = 3;
  static constexpr int kRow = kBlockCh * E + 16;
  static constexpr int kShared = 2 * N * E;
  static constexpr int kStage = T * (4 * kRow + kShared);      // dt, u, dy, z; B and C
  static constexpr int kBC = T * 2 * N * 4;
  static constexpr int kDPart = V * 8 + (V > 2 ? 16 : 0);
  static constexpr int kDRow = kBlockCh / V * kDPart;
  static constexpr int kYRow = kBlockCh * 4 + 32;              // e; a channel's three sums
  static constexpr int kSum = T * 2 * N * 4;                   // dB and dC of a warp's run
  static constexpr size_t kSmem =
      kStages * kStage + 2 * (kBC + T * (kDRow + 4 * kYRow) + kWarps * kSum);
};

template <int DT, int N>
__global__ void __launch_bounds__(2 * kSsmPart, 1)
ssm_bwd_kernel(const SsmParams P) {
  using W = SsmBack<DT, N>;
  using L = SsmLanes<N>;
  constexpr int E = W::E, S = L::kStates, K = L::kPairs, CW = L::kChannels, G = L::kLanes;
  constexpr int T = W::T, V = W::V;
  extern __shared__ __align__(16) char smem[];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == 0 && warp == 0)
    check_cu_seqlens(P.cu_seqlens, P.n_seqs, P.s, P.status);
  const SsmPlace<W::kBlockCh> at(P);
  const int r = at.r;
  const int64_t rc = static_cast<int64_t>(r) * P.c;
  char* bcs = smem + W::kStages * W::kStage;
  char* dds = bcs + 2 * W::kBC;
  char* es = dds + 2 * T * W::kDRow;
  char* outs = es + 2 * T * W::kYRow;                          // [2][3][T] rows of sums
  char* sums = outs + 6 * T * W::kYRow;
  const int64_t row0 = at.batch * P.s + at.tok0;
  const int n_runs = static_cast<int>((at.len + T - 1) / T);
  auto run_of = [&](int k) { return static_cast<int64_t>(n_runs - 1 - k) * T; };
  auto tokens_of = [&](int64_t t0) { return at.len - t0 < T ? static_cast<int>(at.len - t0) : T; };
  const bool gated = P.gated != 0;

  if (warp >= W::kWarps) {
    // ------------------------------------------------------------ preparing --
    const int ht = tid - kSsmPart;
    const char* src[4] = {P.dt[r] + row0 * P.ld_dt + at.ch0 * E,
                          P.u[r] + row0 * P.ld_u + at.ch0 * E,
                          P.dy[r] + row0 * P.ld_dy + at.ch0 * E,
                          gated ? P.z[r] + row0 * P.ld_z + at.ch0 * E : nullptr};
    const char* src_b = P.B[r] + row0 * P.ld_B + at.group * N * E;
    const char* src_c = P.C[r] + row0 * P.ld_C + at.group * N * E;
    const int live_bytes = at.live * E;
    auto ask = [&](int k) {
      char* st = smem + (k % W::kStages) * W::kStage;
      const int64_t t0 = run_of(k);
      const int n_tok = tokens_of(t0);
      constexpr int kPieces = W::kBlockCh * E / 16;
#pragma unroll
      for (int i = ht; i < T * kPieces; i += kSsmPart) {
        const int tok = i / kPieces, p = (i % kPieces) * 16;
        if (tok >= n_tok || p >= live_bytes) continue;
        char* dst = st + tok * W::kRow + p;
        cp_async16(dst, src[0] + (t0 + tok) * P.ld_dt + p);
        cp_async16(dst + T * W::kRow, src[1] + (t0 + tok) * P.ld_u + p);
        cp_async16(dst + 2 * T * W::kRow, src[2] + (t0 + tok) * P.ld_dy + p);
        if (gated) cp_async16(dst + 3 * T * W::kRow, src[3] + (t0 + tok) * P.ld_z + p);
      }
      constexpr int kP = N * E / 16;
      char* sh = st + 4 * T * W::kRow;
#pragma unroll
      for (int i = ht; i < T * kP; i += kSsmPart) {
        const int tok = i / kP, p = (i % kP) * 16;
        if (tok >= n_tok) continue;
        cp_async16(sh + tok * W::kShared + p, src_b + (t0 + tok) * P.ld_B + p);
        cp_async16(sh + tok * W::kShared + N * E + p, src_c + (t0 + tok) * P.ld_C + p);
      }
    };
    const int my = ht / (W::kBlockCh / V), part = ht % (W::kBlockCh / V);
    const bool on = part * V < at.live;
    F2 bias[V / 2], skip[V / 2], dD[V / 2], dbias[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const int64_t c = rc + at.ch0 + part * V + 2 * i;
      bias[i] = on && P.dt_bias != nullptr ? *reinterpret_cast<const F2*>(P.dt_bias + c) : 0;
      skip[i] = on && P.D != nullptr ? *reinterpret_cast<const F2*>(P.D + c) : 0;
      dD[i] = dbias[i] = 0;
    }
    // what is kept of a token's channels until its sums are there
    struct Kept {
      F2 d[V / 2], u[V / 2], e[V / 2], slope[V / 2], dz[V / 2];
    };
    auto prepare = [&](int k, Kept& x) {
      const char* st = smem + (k % W::kStages) * W::kStage + my * W::kRow + part * V * E;
      Pack<DT, V> p;
      lds_pack(p, st);
      unpack_pairs(p, x.d);
      lds_pack(p, st + T * W::kRow);
      unpack_pairs(p, x.u);
      lds_pack(p, st + 2 * T * W::kRow);
      unpack_pairs(p, x.e);
      if (gated) {
        F2 z[V / 2];
        lds_pack(p, st + 3 * T * W::kRow);
        unpack_pairs(p, z);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          // sg = sigmoid(z); silu' = sg (1 + z (1 - sg)), 1 - sg = exp(-z) sg
          // (exp(87) at most, whose reciprocal is normal: no product of infinity and 0)
          const F2 w = exp2_of<DT, DT == SP_F32, -1>(DT == SP_F32 ? z[i] : held_above(z[i], -87.f));
          const F2 sg = rcp2(add2(w, f2(1.f, 1.f)));
          x.dz[i] = mul2(x.e[i], fma2(mul2(z[i], mul2(w, sg)), sg, sg));
          x.e[i] = mul2(x.e[i], mul2(z[i], sg));
        }
      }
      char* dd = dds + ((k & 1) * T + my) * W::kDRow + part * W::kDPart;
      char* ee = es + ((k & 1) * T + my) * W::kYRow + part * V * 4;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        x.d[i] = add2(x.d[i], bias[i]);
        x.slope[i] = f2(1.f, 1.f);
        if (P.softplus) x.d[i] = softplus2<DT>(x.d[i], &x.slope[i]);
        const float2 a = split(x.d[i]), b = split(mul2(x.d[i], x.u[i]));
        *reinterpret_cast<float4*>(dd + 16 * i) = make_float4(a.x, b.x, a.y, b.y);
        *reinterpret_cast<F2*>(ee + 8 * i) = x.e[i];
      }
      const char* sh = smem + (k % W::kStages) * W::kStage + 4 * T * W::kRow;
      float* bc = reinterpret_cast<float*>(bcs + (k & 1) * W::kBC);
#pragma unroll
      for (int i = ht; i < T * 2 * N / 4; i += kSsmPart) {
        Pack<DT, 4> q;
        float f[4];
        lds_pack(q, sh + i * 4 * E);
        unpack(q, f);
        *reinterpret_cast<float4*>(bc + i * 4) = make_float4(f[0], f[1], f[2], f[3]);
      }
    };
    const int live_warps = (at.live + CW - 1) / CW;
    auto finish = [&](int k, const Kept& x) {
      const int64_t t0 = run_of(k);
      const int n_tok = tokens_of(t0);
      // dB and dC: the block's warps in order
      const char* from = sums + (k & 1) * W::kWarps * W::kSum;
#pragma unroll
      for (int i = ht; i < T * 2 * N / 4; i += kSsmPart) {
        const int tok = i / (N / 2), e = (i % (N / 2)) * 4;
        if (tok >= n_tok) continue;
        F2 a = 0, b = 0;
        for (int w = 0; w < live_warps; ++w) {
          const float4 v = *reinterpret_cast<const float4*>(from + w * W::kSum + i * 16);
          a = add2(a, f2(v.x, v.y));
          b = add2(b, f2(v.z, v.w));
        }
        const int64_t row = row0 + t0 + tok;
        if (P.partial_bc != nullptr) {
          const int64_t rows = static_cast<int64_t>(P.b) * P.s;
          const F2 both[2] = {a, b};
          store_states(P.partial_bc + (at.slab * rows + row) * 2 * N + e, both);
        } else {
          Pack<DT, 4> p;
          const F2 both[2] = {a, b};
          pack_pairs(p, both);
          const int n = e % N + at.group * N;
          if (e < N) store_pack(P.dB[r] + row * P.ld_dB + n * E, p);
          else store_pack(P.dC[r] + row * P.ld_dC + n * E, p);
        }
      }
      if (!on || my >= n_tok) return;
      const char* out = outs + ((k & 1) * 3 * T + my) * W::kYRow + part * V * 4;
      F2 du[V / 2], ddt[V / 2], dz[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const F2 through = *reinterpret_cast<const F2*>(out + 8 * i);
        const F2 decay = *reinterpret_cast<const F2*>(out + T * W::kYRow + 8 * i);
        du[i] = fma2(x.d[i], through, mul2(skip[i], x.e[i]));
        ddt[i] = mul2(fma2(x.u[i], through, mul2(decay, f2(kLn2, kLn2))), x.slope[i]);
        if (gated) {
          const F2 inner = *reinterpret_cast<const F2*>(out + 2 * T * W::kYRow + 8 * i);
          dz[i] = mul2(x.dz[i], fma2(skip[i], x.u[i], inner));
        }
        dD[i] = fma2(x.e[i], x.u[i], dD[i]);
        dbias[i] = add2(dbias[i], ddt[i]);
      }
      const int64_t row = row0 + t0 + my, off = (at.ch0 + part * V) * E;
      Pack<DT, V> p;
      pack_pairs(p, du);
      store_pack(P.du[r] + row * P.ld_du + off, p);
      pack_pairs(p, ddt);
      store_pack(P.ddt[r] + row * P.ld_ddt + off, p);
      if (gated) {
        pack_pairs(p, dz);
        store_pack(P.dz[r] + row * P.ld_dz + off, p);
      }
    };
    if (n_runs > 0) ask(0);
    cp_async_commit();
    if (n_runs > 1) ask(1);
    cp_async_commit();
    Kept even, odd;                    // of even and of odd steps
    auto step = [&](int k, Kept& next) {
      cp_async_wait<1>();              // step k + 1's rows
      meet<2 * kSsmPart>();
      // (step k's rows have been prepared: step k + 3 takes their place)
      if (k + 3 < n_runs) ask(k + 3);
      cp_async_commit();
      if (k >= 1) finish(k - 1, next);
      if (k + 1 < n_runs) prepare(k + 1, next);
    };
    if (n_runs > 2) ask(2);
    cp_async_commit();
    cp_async_wait<2>();                // step 0's rows
    meet<2 * kSsmPart>();
    if (n_runs > 0) prepare(0, even);
    for (int k = 0; k <= n_runs; k += 2) {
      step(k, odd);
      if (k + 1 <= n_runs) step(k + 1, even);
    }
    if (P.partial_params == nullptr) return;
    // the block's tokens of a channel, in the order of its threads
    float* to = P.partial_params + (at.batch * P.chunks + at.chunk) * P.t * P.c * (N + 2) +
                static_cast<int64_t>(P.t) * P.c * N;
    F2* sum = reinterpret_cast<F2*>(es);                       // [2][T][kBlockCh / 2]
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      sum[my * (W::kBlockCh / 2) + part * (V / 2) + i] = dD[i];
      sum[(T + my) * (W::kBlockCh / 2) + part * (V / 2) + i] = dbias[i];
    }
    asm volatile("bar.sync 2, %0;" ::"n"(kSsmPart) : "memory");
    if (ht < W::kBlockCh && ht / (W::kBlockCh / 2) < 2) {
      const int which = ht / (W::kBlockCh / 2), c = ht % (W::kBlockCh / 2);
      F2 a = 0;
#pragma unroll
      for (int i = 0; i < T; ++i) a = add2(a, sum[(which * T + i) * (W::kBlockCh / 2) + c]);
      if (2 * c < at.live)
        *reinterpret_cast<F2*>(to + static_cast<int64_t>(which) * P.t * P.c + rc + at.ch0 + 2 * c) = a;
    }
    return;
  }

  // ---------------------------------------------------------------- states --
  const bool active = warp * CW + lane / G * 2 < at.live;
  const int n0 = (lane % G) * S, ch = active ? warp * CW + lane / G * 2 : 0;
  const int64_t mine = (rc + at.ch0 + ch) * N + n0;
  const int64_t state_at = static_cast<int64_t>(at.ch0 + ch) * N + n0;
  const int64_t state_step = static_cast<int64_t>(P.c) * N;
  const int64_t all_runs = (P.s + T - 1) / T;
  const bool packed = P.cu_seqlens != nullptr;
  auto load_both = [&](const float* base, int64_t i, F2 (&x)[2][K]) {
    load_states_or_zero(base, i, x[0]);
    load_states_or_zero(base, i + N, x[1]);
  };
  auto store_both = [&](float* base, int64_t i, const F2 (&x)[2][K]) {
    if (!active) return;
    store_states(base + i, x[0]);
    store_states(base + i + N, x[1]);
  };
  // the gradient that comes from behind (times the decay in between); the decay rates
  // in powers of two, their gradients' sums; the state before the next run
  F2 back[2][K], a2[2][K], dA[2][K], next[2][K];
  load_both(P.A, mine, a2);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int p = 0; p < K; ++p) {
      a2[c][p] = mul2(a2[c][p], f2(kLog2e, kLog2e));
      dA[c][p] = 0;
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
  auto run_state = [&](int k) {
    const int64_t run = (at.tok0 + run_of(k)) / T;
    load_both(P.states[r], (at.batch * all_runs + run) * state_step + state_at, next);
  };
  if (n_runs > 0) run_state(0);
  const int dd_at = ch / V * W::kDPart + ch % V * 8;
  // which of a lane's 2 S sums of dB's and dC's states it keeps, of the 32 / G lanes
  constexpr int CL = 32 / G;
  constexpr int kKept = 2 * S > CL ? 2 * S / CL : 1;
  constexpr int kSame = CL > 2 * S ? CL / (2 * S) : 1;         // lanes with the same
  const int kept = lane / G / kSame * kKept;
  const int put_at = (kept / S) * N + n0 + kept % S;

  meet<2 * kSsmPart>();                // (step 0 is prepared)
  for (int k = 0; k < n_runs; ++k) {
    meet<2 * kSsmPart>();
    const float* shared = reinterpret_cast<const float*>(bcs + (k & 1) * W::kBC) + n0;
    const char* dd = dds + (k & 1) * T * W::kDRow + dd_at;
    const char* ee = es + (k & 1) * T * W::kYRow + ch * 4;
    char* out = outs + (k & 1) * 3 * T * W::kYRow + ch * 4;
    float* put = reinterpret_cast<float*>(sums + ((k & 1) * W::kWarps + warp) * W::kSum) + put_at;
    const int64_t tok0 = at.tok0 + run_of(k);
    const int n_tok = tokens_of(run_of(k));
    F2 first[2][K];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int p = 0; p < K; ++p) first[c][p] = next[c][p];
    if (k + 1 < n_runs) run_state(k + 1);
    SsmMarks marks{0u, 0};
    if (packed) marks = ssm_marks(P, tok0, n_tok);

    // SLOW: runs with less than 16 tokens, or where a sequence begins
    auto go = [&](auto slow) {
      constexpr bool SLOW = decltype(slow)::value;
      constexpr int H = T / 2;
      auto begins = [&](int t) { return SLOW && (marks.starts >> t & 1u); };
      auto forget = [&](int t, F2 (&h)[2][K]) {        // the state before a sequence
        load_both(P.h0[r], __shfl_sync(kAll, marks.seq, t) * state_step + state_at, h);
      };
      // the states after token t, and its decays
      auto token = [&](int t, F2 (&h)[2][K], F2 (&a)[2][K]) {
        const float4 v = *reinterpret_cast<const float4*>(dd + t * W::kDRow);
        const float d[2] = {v.x, v.z}, in[2] = {v.y, v.w};
        F2 b[K];
        load_states(shared + t * 2 * N, b);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int p = 0; p < K; ++p) {
            a[c][p] = pow2(mul2(f2(d[c], d[c]), a2[c][p]));
            h[c][p] = fma2(a[c][p], h[c][p], mul2(f2(in[c], in[c]), b[p]));
          }
      };
      F2 begin[2][K];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int p = 0; p < K; ++p) begin[c][p] = first[c][p];
      if (!SLOW || n_tok > H) {
#pragma unroll
        for (int t = 0; t < H; ++t) {
          F2 a[2][K];
          if (begins(t)) forget(t, begin);
          token(t, begin, a);
        }
      }
#pragma unroll 1
      for (int t0 = H; t0 >= 0; t0 -= H) {
        if (t0 == 0) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int p = 0; p < K; ++p) begin[c][p] = first[c][p];
        }
        F2 h[H][2][K], a[H][2][K], now[2][K];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int p = 0; p < K; ++p) now[c][p] = begin[c][p];
        float inner[8];
#pragma unroll
        for (int i = 0; i < H; ++i) {
          const int t = t0 + i;
          inner[i % 4 * 2] = inner[i % 4 * 2 + 1] = 0.f;
          if (!SLOW || t < n_tok) {
            if (begins(t)) forget(t, now);
            token(t, now, a[i]);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int p = 0; p < K; ++p) h[i][c][p] = now[c][p];
            if (gated) {
              F2 q[K];
              load_states(shared + t * 2 * N + N, q);
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                F2 acc = mul2(now[c][0], q[0]);
                if constexpr (K == 2) acc = fma2(now[c][1], q[1], acc);
                const float2 x = split(acc);
                inner[i % 4 * 2 + c] = x.x + x.y;
              }
            }
          }
          if (gated && i % 4 == 3) {
            sum_over<8, G>(inner, lane, 1);
            constexpr int kEach = G >= 8 ? 1 : 8 / G;
            const int id = (lane % G) / (G >= 8 ? G / 8 : 1) * kEach;  // token 2, channel 1
            char* dst = out + (2 * T + t - 3 + id / 2) * W::kYRow + id % 2 * 4;
            if (active) {
              if constexpr (kEach == 2) *reinterpret_cast<float2*>(dst) = make_float2(inner[0], inner[1]);
              else *reinterpret_cast<float*>(dst) = inner[0];
            }
          }
        }
        float part[16];
#pragma unroll
        for (int i = H - 1; i >= 0; --i) {
          const int t = t0 + i;
          float* sum4 = part + i % 4 * 4;              // of a token: through, decay; channels
          sum4[0] = sum4[1] = sum4[2] = sum4[3] = 0.f;
          if (!SLOW || t < n_tok) {
            const float4 x = *reinterpret_cast<const float4*>(dd + t * W::kDRow);
            const float2 ev = *reinterpret_cast<const float2*>(ee + t * W::kYRow);
            const float d[2] = {x.x, x.z}, in[2] = {x.y, x.w}, e[2] = {ev.x, ev.y};
            F2 b[K], q[K], db[K], dc[K], before[2][K];
            load_states(shared + t * 2 * N, b);
            load_states(shared + t * 2 * N + N, q);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int p = 0; p < K; ++p)
                before[c][p] = i > 0 ? h[i > 0 ? i - 1 : 0][c][p] : begin[c][p];
            if (begins(t)) forget(t, before);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const F2 e2 = f2(e[c], e[c]), in2 = f2(in[c], in[c]), d2 = f2(d[c], d[c]);
              F2 through = 0, decay = 0;
#pragma unroll
              for (int p = 0; p < K; ++p) {
                const F2 gr = fma2(q[p], e2, back[c][p]);
                dc[p] = c == 0 ? mul2(h[i][c][p], e2) : fma2(h[i][c][p], e2, dc[p]);
                db[p] = c == 0 ? mul2(gr, in2) : fma2(gr, in2, db[p]);
                through = p == 0 ? mul2(gr, b[p]) : fma2(gr, b[p], through);
                back[c][p] = mul2(a[i][c][p], gr);
                const F2 g = mul2(back[c][p], before[c][p]);
                decay = p == 0 ? mul2(g, a2[c][p]) : fma2(g, a2[c][p], decay);
                dA[c][p] = fma2(g, d2, dA[c][p]);
              }
              const float2 y = split(through), w = split(decay);
              sum4[c] = y.x + y.y;
              sum4[2 + c] = w.x + w.y;
            }
            if (begins(t)) {
              const int64_t seq = __shfl_sync(kAll, marks.seq, t);
              if (P.hT[r] != nullptr) store_both(P.hT[r], seq * state_step + state_at, back);
              const float* from = tok0 + t > 0 ? P.dhT[r] : nullptr;
              const int64_t prev =
                  tok0 + t > 0 ? find_seq(P.cu_seqlens, P.n_seqs, tok0 + t - 1) : 0;
              load_both(from, prev * state_step + state_at, back);
            }
            float v[2 * S];
#pragma unroll
            for (int p = 0; p < K; ++p) {
              const float2 y = split(db[p]), w = split(dc[p]);
              v[2 * p] = active ? y.x : 0.f;
              v[2 * p + 1] = active ? y.y : 0.f;
              v[S + 2 * p] = active ? w.x : 0.f;
              v[S + 2 * p + 1] = active ? w.y : 0.f;
            }
            sum_over<2 * S, CL>(v, lane, G);
#pragma unroll
            for (int j = 0; j < kKept; ++j) put[t * 2 * N + j] = v[j];
          }
          if (i % 4 == 0) {
            sum_over<16, G>(part, lane, 1);
            constexpr int kEach = 16 / G;
            const int id = lane % G * kEach;           // token 4, sum 2, channel 1
            char* dst = out + (t + id / 4) * W::kYRow;
            if (active) {
              if constexpr (kEach == 4) {
                *reinterpret_cast<float2*>(dst) = make_float2(part[0], part[1]);
                *reinterpret_cast<float2*>(dst + T * W::kYRow) = make_float2(part[2], part[3]);
              } else if constexpr (kEach == 2) {
                *reinterpret_cast<float2*>(dst + id / 2 % 2 * T * W::kYRow) =
                    make_float2(part[0], part[1]);
              } else {
                *reinterpret_cast<float*>(dst + id / 2 % 2 * T * W::kYRow + id % 2 * 4) = part[0];
              }
            }
          }
        }
      }
    };
    if (marks.starts == 0u && n_tok == T) go(std::false_type{});
    else go(std::true_type{});
  }
  meet<2 * kSsmPart>();                // (the preparers finish the last step)
  if (!packed && at.chunk == 0 && P.hT[r] != nullptr)
    store_both(P.hT[r], at.batch * state_step + state_at, back);
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
__global__ void __launch_bounds__(kPartThreads)
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
  const void* fn = reinterpret_cast<const void*>(&ssm_bwd_kernel<DT, N>);
  const cudaError_t e = ensure_smem_attr(fn, W::kSmem);
  if (e != cudaSuccess) return e;
  void* args[] = {const_cast<SsmParams*>(&p)};
  const int64_t grid = static_cast<int64_t>(p.b) * p.chunks * p.t * p.groups * p.slabs;
  return launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(2 * kSsmPart), W::kSmem, args, st);
}

}  // namespace spb
