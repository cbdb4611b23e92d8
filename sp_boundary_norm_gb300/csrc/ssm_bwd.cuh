// Selective scan, backward.  With e = dy silu(z), along the tokens from the last:
//   G[i] = C[i] e[i] + a[i+1] G[i+1],   a = exp(d A)
//   dC[i] = sum over a group's channels of e h,  dB[i] = the same of G d u
//   g = a G h[i-1],   d(d u) = sum_n G B,   d(d) = sum_n g A + u d(d u)
//   dA = sum over tokens of g d
// A block takes the channels of eight warps and walks its chunk from the end, a run of
// 16 tokens a step: it starts from the state that the forward saved for the run, goes
// through the run once forwards, keeping the 16 states and decays in registers, and
// once backwards.  dB and dC of a token are summed over a warp's lanes, then over the
// block's warps in shared memory, then by a second kernel over the blocks of a
// group's channels: always in the same order.
#include <type_traits>

#include "ssm.cuh"

namespace spb {

template <int DT, int N>
struct SsmBack {
  using L = SsmLanes<N>;
  static constexpr int kWarps = 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kBlockCh = kWarps * L::kChannels;
  static constexpr int E = ElemSize<DT>::value;
  static constexpr int R = kSsmRun;
  static constexpr int kStages = 3;
  static constexpr int kRow = kBlockCh * E + 16;
  static constexpr int kShared = 2 * N * E;
  static constexpr int kStage = R * (4 * kRow + kShared);      // dt, u, dy, z; B and C
  static constexpr int kBC = R * 2 * N * 4;
  static constexpr int kDRow = L::kChannels * 16 + 16;
  static constexpr int kFRow = L::kChannels * 4 + 16;
  // of a warp: (d, d, d u, d u), (e, e, u, slope), and four floats a token and channel
  static constexpr int kOwn = R * (2 * kDRow + 4 * kFRow);
  static constexpr int kSum = R * 2 * N * 4;                   // dB and dC of a warp's run
  static constexpr int kParam = kBlockCh * 2 * 4;
  static constexpr size_t kSmem =
      kStages * kStage + 2 * kBC + kWarps * kOwn + 2 * kWarps * kSum + kParam;
};

template <int DT, int N>
__global__ void __launch_bounds__(SsmBack<DT, N>::kThreads, 1)
ssm_bwd_kernel(const SsmParams P) {
  using W = SsmBack<DT, N>;
  using L = SsmLanes<N>;
  constexpr int E = W::E, K = L::kPairs, S = L::kStates, CW = L::kChannels, G = L::kLanes;
  constexpr int R = W::R, V = CW / 2;  // channels of a lane's token
  extern __shared__ __align__(16) char smem[];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x == 0 && warp == 0)
    check_cu_seqlens(P.cu_seqlens, P.n_seqs, P.s, P.status);
  const SsmPlace<W::kBlockCh> at(P);
  const int r = at.r;
  const int64_t rc = static_cast<int64_t>(r) * P.c;
  char* bc = smem + W::kStages * W::kStage;
  char* own = bc + 2 * W::kBC + warp * W::kOwn;
  char* aux = own + R * W::kDRow;
  char* flo = aux + R * W::kDRow;                              // four [R][kFRow]
  char* sums = bc + 2 * W::kBC + W::kWarps * W::kOwn;
  float* param = reinterpret_cast<float*>(sums + 2 * W::kWarps * W::kSum);
  for (int i = tid; i < W::kBlockCh; i += W::kThreads) {
    const bool on = i < at.live;
    param[i] = on && P.dt_bias != nullptr ? P.dt_bias[rc + at.ch0 + i] : 0.f;
    param[W::kBlockCh + i] = on && P.D != nullptr ? P.D[rc + at.ch0 + i] : 0.f;
  }
  const int64_t row0 = at.batch * P.s + at.tok0;
  const char* src[4] = {P.dt[r] + row0 * P.ld_dt + at.ch0 * E,
                        P.u[r] + row0 * P.ld_u + at.ch0 * E,
                        P.dy[r] + row0 * P.ld_dy + at.ch0 * E,
                        P.gated ? P.z[r] + row0 * P.ld_z + at.ch0 * E : nullptr};
  const char* src_b = P.B[r] + row0 * P.ld_B + at.group * N * E;
  const char* src_c = P.C[r] + row0 * P.ld_C + at.group * N * E;
  const bool gated = P.gated != 0;
  const int n_runs = static_cast<int>((at.len + R - 1) / R);
  const int live_bytes = at.live * E;
  auto ask = [&](int k) {
    char* st = smem + (k % W::kStages) * W::kStage;
    const int64_t t0 = static_cast<int64_t>(n_runs - 1 - k) * R;
    const int n_tok = at.len - t0 < R ? static_cast<int>(at.len - t0) : R;
    constexpr int kPieces = W::kBlockCh * E / 16;
#pragma unroll
    for (int i = tid; i < R * kPieces; i += W::kThreads) {
      const int tok = i / kPieces, p = (i % kPieces) * 16;
      if (tok >= n_tok || p >= live_bytes) continue;
      char* dst = st + tok * W::kRow + p;
      cp_async16(dst, src[0] + (t0 + tok) * P.ld_dt + p);
      cp_async16(dst + R * W::kRow, src[1] + (t0 + tok) * P.ld_u + p);
      cp_async16(dst + 2 * R * W::kRow, src[2] + (t0 + tok) * P.ld_dy + p);
      if (gated) cp_async16(dst + 3 * R * W::kRow, src[3] + (t0 + tok) * P.ld_z + p);
    }
    constexpr int kP = N * E / 16;
    char* sh = st + 4 * R * W::kRow;
    for (int i = tid; i < n_tok * kP; i += W::kThreads) {
      const int tok = i / kP, p = (i - tok * kP) * 16;
      cp_async16(sh + tok * W::kShared + p, src_b + (t0 + tok) * P.ld_B + p);
      cp_async16(sh + tok * W::kShared + N * E + p, src_c + (t0 + tok) * P.ld_C + p);
    }
  };
  auto widen = [&](int k) {
    const char* sh = smem + (k % W::kStages) * W::kStage + 4 * R * W::kRow;
    float* dst = reinterpret_cast<float*>(bc + (k & 1) * W::kBC);
    for (int i = tid; i < R * 2 * N / 4; i += W::kThreads) {
      Pack<DT, 4> p;
      float f[4];
      lds_pack(p, sh + i * 4 * E);
      unpack(p, f);
      *reinterpret_cast<float4*>(dst + i * 4) = make_float4(f[0], f[1], f[2], f[3]);
    }
  };
  // step k's dB and dC: the block's warps in order
  const int live_warps = at.live / CW;
  auto put_bc = [&](int k) {
    const int64_t t0 = static_cast<int64_t>(n_runs - 1 - k) * R;
    const int n_tok = at.len - t0 < R ? static_cast<int>(at.len - t0) : R;
    const float* from = reinterpret_cast<const float*>(sums + (k & 1) * W::kWarps * W::kSum);
    for (int i = tid; i < n_tok * 2 * N / 4; i += W::kThreads) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < live_warps; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(from + w * R * 2 * N + i * 4);
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
      const int tok = i / (N / 2), e = i - tok * (N / 2);
      const int64_t row = row0 + t0 + tok;
      if (P.partial_bc != nullptr) {
        const int64_t rows = static_cast<int64_t>(P.b) * P.s;
        *reinterpret_cast<float4*>(P.partial_bc + (at.slab * rows + row) * 2 * N + e * 4) = a;
      } else {
        Pack<DT, 4> p;
        const float f[4] = {a.x, a.y, a.z, a.w};
        pack(p, f);
        const int n = e * 4 % N + at.group * N;
        if (e * 4 < N) store_pack(P.dB[r] + row * P.ld_dB + n * E, p);
        else store_pack(P.dC[r] + row * P.ld_dC + n * E, p);
      }
    }
  };

  const bool active = warp * CW < at.live;
  const int n0 = (lane % G) * S, ch = warp * CW + lane / G;
  const int64_t mine = (rc + at.ch0 + ch) * N + n0;
  const int64_t state_at = static_cast<int64_t>(at.ch0 + ch) * N + n0;
  const int64_t state_step = static_cast<int64_t>(P.c) * N;
  const int64_t all_runs = (P.s + R - 1) / R;
  const bool packed = P.cu_seqlens != nullptr;
  // the gradient that comes from behind (times the decay in between), the decay
  // rates in powers of two, their gradient's sums
  F2 back[K], a2[K], dA[K], first[K];
  float dD[V], dbias[V];
  clear(back);
  clear(a2);
  clear(dA);
  clear(first);
#pragma unroll
  for (int i = 0; i < V; ++i) dD[i] = dbias[i] = 0.f;
  auto run_state = [&](int64_t t0, F2 (&x)[K]) {
    const int64_t run = (at.tok0 + t0) / R;
    load_states(P.states[r] + (at.batch * all_runs + run) * state_step + state_at, x);
  };
  if (active) {
    load_states(P.A + mine, a2);
#pragma unroll
    for (int p = 0; p < K; ++p) a2[p] = mul2(a2[p], f2(kLog2e, kLog2e));
    if (P.chunks > 1) {
      load_states(P.carry + (at.batch * P.chunks + at.chunk) * P.t * P.c * N + mine, back);
    } else {
      const int64_t seq = packed ? find_seq(P.cu_seqlens, P.n_seqs, P.s - 1) : at.batch;
      load_states_or_zero(P.dhT[r], seq * state_step + state_at, back);
    }
    if (packed && at.chunk == 0 && P.hT[r] != nullptr) {
      // the gradients of the states of sequences without a token pass
      for (int j = 0; j < P.n_seqs; ++j) {
        if (__ldg(P.cu_seqlens + j) != __ldg(P.cu_seqlens + j + 1)) continue;
        F2 v[K];
        load_states_or_zero(P.dhT[r], j * state_step + state_at, v);
        store_states(P.hT[r] + j * state_step + state_at, v);
      }
    }
    if (n_runs > 0) run_state(static_cast<int64_t>(n_runs - 1) * R, first);
  }

  if (n_runs > 0) ask(0);
  cp_async_commit();
  if (n_runs > 1) ask(1);
  cp_async_commit();
  cp_async_wait<1>();
  __syncthreads();
  if (n_runs > 0) widen(0);
  for (int k = 0; k < n_runs; ++k) {
    cp_async_wait<0>();
    __syncthreads();                   // step k + 1's rows, step k's B and C, k - 1's sums
    if (k + 2 < n_runs) ask(k + 2);
    cp_async_commit();
    if (k + 1 < n_runs) widen(k + 1);
    if (k > 0) put_bc(k - 1);
    if (!active) continue;
    const char* st = smem + (k % W::kStages) * W::kStage + warp * CW * E;
    const float* shared = reinterpret_cast<const float*>(bc + (k & 1) * W::kBC) + n0;
    const int64_t t0 = static_cast<int64_t>(n_runs - 1 - k) * R, tok0 = at.tok0 + t0;
    const int n_tok = at.len - t0 < R ? static_cast<int>(at.len - t0) : R;
    F2 start_state[K];
#pragma unroll
    for (int p = 0; p < K; ++p) start_state[p] = first[p];
    if (k + 1 < n_runs) run_state(t0 - R, first);

    // a lane prepares one token of half the warp's channels
    const int my = lane % R, half = lane / R * V;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      constexpr int M = V >= 2 ? 2 : 1;
      const char* at_ch = st + my * W::kRow + (half + i) * E;
      Pack<DT, M> p;
      float f[4][2];
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        if (a == 3 && !gated) continue;
        float x[M];
        lds_pack(p, at_ch + a * R * W::kRow);
        unpack(p, x);
        f[a][0] = x[0];
        f[a][1] = x[M - 1];
      }
      F2 d = f2(f[0][0] + param[warp * CW + half + i], f[0][1] + param[warp * CW + half + i + M - 1]);
      const F2 u = f2(f[1][0], f[1][1]), dy = f2(f[2][0], f[2][1]);
      F2 slope = f2(1.f, 1.f), e = dy, dz = 0;
      if (P.softplus) d = softplus2<DT>(d, &slope);
      if (gated) {
        const F2 z = f2(f[3][0], f[3][1]);
        const F2 x = exp2_of<DT, DT == SP_F32, -1>(DT == SP_F32 ? z : held_above(z, -87.f));
        const F2 sg = rcp2(add2(x, f2(1.f, 1.f)));
        e = mul2(dy, mul2(z, sg));
        // silu' = sg (1 + z (1 - sg)), 1 - sg = x sg
        dz = mul2(dy, fma2(mul2(z, mul2(x, sg)), sg, sg));
      }
      const float2 dd = split(d), du = split(mul2(d, u)), uu = split(u), ee = split(e);
      const float2 ss = split(slope), zz = split(dz);
#pragma unroll
      for (int j = 0; j < M; ++j) {
        const int c = half + i + j;
        const float dv = j ? dd.y : dd.x, duv = j ? du.y : du.x, ev = j ? ee.y : ee.x;
        *reinterpret_cast<float4*>(own + my * W::kDRow + c * 16) = make_float4(dv, dv, duv, duv);
        *reinterpret_cast<float4*>(aux + my * W::kDRow + c * 16) =
            make_float4(ev, ev, j ? uu.y : uu.x, j ? ss.y : ss.x);
        *reinterpret_cast<float*>(flo + 3 * R * W::kFRow + my * W::kFRow + c * 4) =
            j ? zz.y : zz.x;
      }
    }
    __syncwarp();

    SsmMarks marks{0u, 0};
    if (packed) marks = ssm_marks(P, tok0, n_tok);
    const int lc = lane / G;
    float* put = reinterpret_cast<float*>(sums + ((k & 1) * W::kWarps + warp) * W::kSum);
    constexpr int kKept = 2 * S / CW > 1 ? 2 * S / CW : 1;     // sums of dB and dC a lane keeps
    constexpr int kPart = 2 * S >= CW ? CW : 2 * S;            // parts that they are cut into
    // the first of a lane's kept sums, of the lane's 2 S values (dB's states, dC's)
    const int kept = lc / (CW / kPart) * kKept;
    const int put_at = (kept / S) * N + n0 + kept % S;

    // SLOW: runs with less than 16 tokens, or where a sequence begins
    auto go = [&](auto slow) {
      constexpr bool SLOW = decltype(slow)::value;
      F2 h[R][K], a[R][K];
      F2 now[K];
#pragma unroll
      for (int p = 0; p < K; ++p) now[p] = start_state[p];
      float inner[4];
#pragma unroll
      for (int t = 0; t < R; ++t) {
        inner[t % 4] = 0.f;
        if (!SLOW || t < n_tok) {
          if (SLOW && (marks.starts >> t & 1u))
            load_states_or_zero(P.h0[r], __shfl_sync(kAll, marks.seq, t) * state_step + state_at, now);
          const float4 d = *reinterpret_cast<const float4*>(own + t * W::kDRow + lc * 16);
          const F2 step = f2(d.x, d.y), in = f2(d.z, d.w);
          F2 b[K];
          load_states(shared + t * 2 * N, b);
#pragma unroll
          for (int p = 0; p < K; ++p) {
            a[t][p] = pow2(mul2(step, a2[p]));
            now[p] = fma2(a[t][p], now[p], mul2(in, b[p]));
            h[t][p] = now[p];
          }
          if (gated) {
            F2 c[K];
            load_states(shared + t * 2 * N + N, c);
            F2 acc = mul2(now[0], c[0]);
            if constexpr (K == 2) acc = fma2(now[1], c[1], acc);
            const float2 v = split(acc);
            inner[t % 4] = v.x + v.y;
          }
        }
        if (gated && t % 4 == 3) {
          sum_over<4, G>(inner, lane, 1);
          // lanes that hold the same sum write it together
          *reinterpret_cast<float*>(flo + 2 * R * W::kFRow +
                                    (t - 3 + (lane % G) / (G / 4)) * W::kFRow + lc * 4) = inner[0];
        }
      }
      float part[8];
#pragma unroll
      for (int t = R - 1; t >= 0; --t) {
        part[t % 4] = part[4 + t % 4] = 0.f;
        if (!SLOW || t < n_tok) {
          const float4 d = *reinterpret_cast<const float4*>(own + t * W::kDRow + lc * 16);
          const float2 ev = *reinterpret_cast<const float2*>(aux + t * W::kDRow + lc * 16);
          const F2 step = f2(d.x, d.y), in = f2(d.z, d.w), e = f2(ev.x, ev.y);
          F2 b[K], c[K], prev[K];
          load_states(shared + t * 2 * N, b);
          load_states(shared + t * 2 * N + N, c);
          const bool start = SLOW && (marks.starts >> t & 1u);
#pragma unroll
          for (int p = 0; p < K; ++p) prev[p] = t > 0 ? h[t > 0 ? t - 1 : 0][p] : start_state[p];
          int64_t seq = 0;
          if (start) {
            seq = __shfl_sync(kAll, marks.seq, t);
            load_states_or_zero(P.h0[r], seq * state_step + state_at, prev);
          }
          float v[2 * S];
          F2 through = 0, decay = 0;
#pragma unroll
          for (int p = 0; p < K; ++p) {
            const F2 gr = fma2(c[p], e, back[p]);
            const float2 dc = split(mul2(h[t][p], e)), db = split(mul2(gr, in));
            v[2 * p] = db.x;
            v[2 * p + 1] = db.y;
            v[S + 2 * p] = dc.x;
            v[S + 2 * p + 1] = dc.y;
            through = p == 0 ? mul2(gr, b[p]) : fma2(gr, b[p], through);
            back[p] = mul2(a[t][p], gr);
            const F2 g = mul2(back[p], prev[p]);
            decay = p == 0 ? mul2(g, a2[p]) : fma2(g, a2[p], decay);
            dA[p] = fma2(g, step, dA[p]);
          }
          if (start) {
            if (P.hT[r] != nullptr) store_states(P.hT[r] + seq * state_step + state_at, back);
            const int64_t tok = tok0 + t;
            if (tok > 0)
              load_states_or_zero(P.dhT[r],
                                  find_seq(P.cu_seqlens, P.n_seqs, tok - 1) * state_step + state_at,
                                  back);
            else clear(back);
          }
          const float2 x = split(through), y = split(decay);
          part[t % 4] = x.x + x.y;
          part[4 + t % 4] = y.x + y.y;
          sum_over<2 * S, CW>(v, lane, G);
#pragma unroll
          for (int i = 0; i < kKept; ++i) put[t * 2 * N + put_at + i] = v[i];
        }
        if (t % 4 == 0) {
          // two sums of four tokens over a channel's lanes
          sum_over<8, G>(part, lane, 1);
          constexpr int kEach = G >= 8 ? 1 : 8 / G;
          const int id = (lane % G) / (G >= 8 ? G / 8 : 1) * kEach;
#pragma unroll
          for (int i = 0; i < kEach; ++i)
            *reinterpret_cast<float*>(flo + (id / 4) * R * W::kFRow +
                                      (t + id % 4 + i) * W::kFRow + lc * 4) = part[i];
        }
      }
    };
    if (marks.starts == 0u && n_tok == R) go(std::false_type{});
    else go(std::true_type{});
    __syncwarp();

    // a lane finishes one token of half the warp's channels
    float du[V], ddt[V], dz[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = half + i;
      const float4 d = *reinterpret_cast<const float4*>(own + my * W::kDRow + c * 16);
      const float4 x = *reinterpret_cast<const float4*>(aux + my * W::kDRow + c * 16);
      const float* f = reinterpret_cast<const float*>(flo + my * W::kFRow + c * 4);
      constexpr int kF = R * W::kFRow / 4;
      const float through = f[0], decay = f[kF] * kLn2, skip = param[W::kBlockCh + warp * CW + c];
      du[i] = fmaf(d.x, through, skip * x.x);
      ddt[i] = fmaf(x.z, through, decay) * x.w;
      if (gated) dz[i] = f[3 * kF] * fmaf(skip, x.z, f[2 * kF]);
      if (my < n_tok) {
        dD[i] = fmaf(x.x, x.z, dD[i]);
        dbias[i] += ddt[i];
      }
    }
    if (my < n_tok) {
      const int64_t row = row0 + t0 + my;
      const int64_t off = (at.ch0 + warp * CW + half) * E;
      Pack<DT, V> p;
      pack(p, du);
      store_pack(P.du[r] + row * P.ld_du + off, p);
      pack(p, ddt);
      store_pack(P.ddt[r] + row * P.ld_ddt + off, p);
      if (gated) {
        pack(p, dz);
        store_pack(P.dz[r] + row * P.ld_dz + off, p);
      }
    }
  }
  __syncthreads();
  if (n_runs > 0) put_bc(n_runs - 1);
  if (!active) return;
  if (!packed && at.chunk == 0 && P.hT[r] != nullptr)
    store_states(P.hT[r] + at.batch * state_step + state_at, back);
  if (P.partial_params != nullptr) {
    float* to = P.partial_params +
                (at.batch * P.chunks + at.chunk) * P.t * P.c * (N + 2);
    const int64_t all = static_cast<int64_t>(P.t) * P.c;
    store_states(to + mine, dA);
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int m = R / 2; m > 0; m /= 2) {
        dD[i] += __shfl_xor_sync(kAll, dD[i], m);
        dbias[i] += __shfl_xor_sync(kAll, dbias[i], m);
      }
      if (lane % R == 0) {
        const int64_t c = rc + at.ch0 + warp * CW + lane / R * V + i;
        to[all * N + c] = dD[i];
        to[all * (N + 1) + c] = dbias[i];
      }
    }
  }
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

// The parameters' gradients: the blocks of a channel in order.
__global__ void __launch_bounds__(256)
ssm_params_kernel(const float* from, int64_t channels, int n, int64_t parts, SsmParamGrads g) {
  pdl_wait();
  const int64_t all = channels * (n + 2);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= all) return;
  float a = 0.f;
#pragma unroll 8
  for (int64_t k = 0; k < parts; ++k) a += from[k * all + i];
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
  return launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(W::kThreads), W::kSmem, args, st);
}

}  // namespace spb
