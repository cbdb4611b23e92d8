// Causal convolution, backward:
//   dq[i] = dy[i] act'(q[i]),  dx[i] = sum_j w[j] dq[i + W - 1 - j] inside a sequence
//   dw[j] = sum_i dq[i] x[i - (W - 1) + j],  dbias = sum_i dq[i]
// A thread walks runs of tokens of its channels: q is computed again from the
// inputs, and each token's gradient is added to those of the W - 1 tokens before it,
// which wait in registers until they are whole.  A run goes on for W - 1 tokens beyond
// its end for the gradients that come from there.  The parameters' sums of 128 tokens stay
// in registers; a thread's, a block's and (by sum_parts) all blocks' are added up from them,
// always in the same order.
//
// Bound by reading x and dy and writing dx: on a GB300, bf16, 8 ranks' 16,384 x 1024 with
// four taps and silu, 805 MB in 155 us, 5.2 TB/s; per channel and token two reciprocals,
// two exponentials and 13 products are then on their way in 16 warps an SM.  Two channels a
// thread, for twice the warps, took a third longer (every load is half as wide); five
// blocks an SM spilled and took 30 % longer.
#include "conv.cuh"

namespace spb {

constexpr int kConvBlocksB = 4;        // of an SM, by their registers
// Tokens that are added one by one before their sums join the others, in local memory.  (One
// sum for all of a thread's tokens, as many as a call has for its channels, loses digits with
// their number: 4096 of them 4e-7 in norm, so 1e-7.  8 ranks' 16,384 x 1024, both
// directions: 235 us and dweight off by 3.9e-7, every 128 tokens 240 and 2.2e-7, every 64 241
// and 1.8e-7; with the other sums in registers 248.)
constexpr int kSumTokens = 128;

// Where a run's gradients go; this lane's channels.
template <int V>
struct RowOut {
  char* dx;            // of the run's first token
  char* dx0;           // of the call's first state, or NULL
  const char* dxT;     // of its gradient, or NULL
  int64_t ld, state;   // bytes between tokens, and between the rows of a state
  int n;               // tokens of the run
};

// The gradient of the run's token `row`, or of the row of q's state that stands for it,
// is whole: not the run's own are left out.  (Its own code, which few rows come to.)
template <int DT, int V, int W>
__device__ __noinline__ void put_row(RowOut<V> out, ConvSeq q, int row, F2 a, F2 b) {
  static_assert(V == 4, "two pairs");
  if (row >= out.n || (row < 0 && (row >= q.lo || q.lo < 0))) return;
  char* dst;
  if (row >= q.lo) dst = out.dx + row * out.ld;
  else if (out.dx0 != nullptr)
    dst = out.dx0 + (static_cast<int64_t>(q.id) * (W - 1) + (W - 1 + row - q.lo)) * out.state;
  else return;
  F2 o[2] = {a, b};
  Pack<DT, V> p;
  if (out.dxT != nullptr && row >= q.hi - (W - 1)) {
    load_pack(p, out.dxT + (static_cast<int64_t>(q.id) * (W - 1) + (row - q.hi + W - 1)) * out.state);
    F2 more[2];
    unpack_pairs(p, more);
    o[0] = add2(o[0], more[0]);
    o[1] = add2(o[1], more[1]);
  }
  pack_pairs(p, o);
  store_pack(dst, p);
}

template <int DT, int W, bool PACKED>
__global__ void __launch_bounds__(kConvThreads, kConvBlocksB)
conv_bwd_kernel(const ConvParams P) {
  constexpr int V = kConvVec, K = V / 2, E = ElemSize<DT>::value, S = V * (W + 1);
  constexpr int U = kConvGroup;
  using Ring = RowRing<DT, V, 2>;
  constexpr int kSums = kConvThreads * (S + 1) * 4;
  __shared__ __align__(16) char space[Ring::kSize > kSums ? Ring::kSize : kSums];
  pdl_wait();
  if (PACKED && blockIdx.x == 0 && threadIdx.x < 32)
    check_cu_seqlens(P.cu_seqlens, P.n_seqs, P.s, P.status);
  const int slots = kConvThreads / P.lanes;
  const int lane = threadIdx.x % P.lanes, slot = threadIdx.x / P.lanes;
  const int part = blockIdx.x / P.slabs, slab = blockIdx.x % P.slabs;
  const int per_rank = P.slabs / P.t;
  const int r = slab / per_rank, vec = (slab - r * per_rank) * P.lanes + lane;
  const bool on = vec < P.vecs;
  const int64_t ch = static_cast<int64_t>(r) * P.c + (on ? vec : 0) * V;
  const int64_t off = (on ? vec : 0) * V * E;
  const char* x0 = P.x0[r] != nullptr ? P.x0[r] + off : nullptr;
  const char* dxT = P.dxT[r] != nullptr ? P.dxT[r] + off : nullptr;
  char* dx0 = P.xT[r] != nullptr ? P.xT[r] + off : nullptr;
  Taps<DT, V, W> taps;
  taps.load(P, ch);
  // the parameters' gradients: the last tokens', and in local memory those before them
  F2 dw[W][K], db[K], whole[W + 1][K];
  auto take_up = [&] {
    asm volatile("" ::"l"(&whole) : "memory");
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        whole[j][k] = add2(whole[j][k], dw[j][k]);
        dw[j][k] = 0;
      }
      whole[W][k] = add2(whole[W][k], db[k]);
      db[k] = 0;
    }
    asm volatile("" ::"l"(&whole) : "memory");
  };
#pragma unroll
  for (int k = 0; k < K; ++k) {
    db[k] = whole[W][k] = 0;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][k] = whole[j][k] = 0;
  }
  const int64_t all = P.runs * P.b;
  for (int64_t at = static_cast<int64_t>(part) * slots + slot; on && at < all;
       at += static_cast<int64_t>(P.parts) * slots) {
    const int64_t batch = divide(at, P.runs, all), i0 = (at - batch * P.runs) * P.run;
    const int n = i0 + P.run < P.s ? P.run : static_cast<int>(P.s - i0);
    const int all_n = i0 + n + W - 1 < P.s ? n + W - 1 : static_cast<int>(P.s - i0);
    const char* x = P.x[r] + (batch * P.s + i0) * P.ld_x + off;
    const char* dy = P.dy[r] + (batch * P.s + i0) * P.ld_dy + off;
    char* dx = P.out[r] + (batch * P.s + i0) * P.ld_out + off;
    Ring ring(space);
    ring.src[0] = x;
    ring.src[1] = dy;
    ring.ld[0] = P.ld_x;
    ring.ld[1] = P.ld_dy;
    cp_async_wait<0>();
#pragma unroll
    for (int g = 0; g < kConvAhead; ++g) ring.ask(all_n - g * U);
    ConvSeq q = conv_seq<PACKED>(P, batch, i0, 0);
    F2 win[W - 1][K], wait[W - 1][K];
    load_window<DT, V, W>(P, x, x0, q, 0, win);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int k = 0; k < K; ++k) wait[j][k] = 0;

    const RowOut<V> out{dx, dx0, dxT, P.ld_out, static_cast<int64_t>(P.c) * E, n};
    auto emit = [&](int row, const F2 (&v)[K]) { put_row<DT, V, W>(out, q, row, v[0], v[1]); };
    auto flush = [&](int end) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) emit(end - (W - 1) + j, wait[j]);
    };

    // One token: its gradient joins the parameters' (OWN) and those of the tokens before
    // it, of which the one W - 1 back is whole.
    auto one = [&](int u, bool own, F2 (&done)[K]) {
      Pack<DT, V> p;
      F2 v[K], g[K], o[K];
      ring.row(u, 0, p);
      unpack_pairs(p, v);
      ring.row(u, 1, p);
      unpack_pairs(p, g);
      if (P.act == SP_ACT_SILU) {
        taps.apply(win, v, o);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          // sigmoid + silu (1 - sigmoid)
          const F2 sg = rcp2(add2(exp2_of<DT, false, -1>(o[k]), f2(1.f, 1.f)));
          g[k] = mul2(g[k], fma2(mul2(o[k], sg), fma2(sg, f2(-1.f, -1.f), f2(1.f, 1.f)), sg));
        }
      }
      if (own) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          db[k] = add2(db[k], g[k]);
#pragma unroll
          for (int j = 0; j < W - 1; ++j) dw[j][k] = fma2(g[k], win[j][k], dw[j][k]);
          dw[W - 1][k] = fma2(g[k], v[k], dw[W - 1][k]);
        }
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        done[k] = fma2(taps.w[0][k], g[k], wait[0][k]);
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j)
          wait[j][k] = fma2(taps.w[j + 1][k], g[k], wait[j + 1][k]);
        wait[W - 2][k] = mul2(taps.w[W - 1][k], g[k]);
      }
      shift<W, K>(win, v);
    };
    // Groups of rows from `lo` on and before `hi` are whole tokens of the run and of one
    // sequence, stored as they are.
    auto group_lo = [&] { return (q.lo > 0 ? q.lo : 0) + W - 1; };
    auto group_hi = [&] { return (q.hi < n ? q.hi : n) - U; };
    int lo = group_lo(), hi = group_hi();
    char* to = dx - (W - 1) * P.ld_out;
    bool open = true;
    for (int i = 0; open && i < all_n; i += U) {
      ring.ask(all_n - i - kConvAhead * U);
      cp_async_wait<kConvAhead>();
      if (i >= lo && i <= hi) {
#pragma unroll
        for (int u = 0; u < U; ++u, to += P.ld_out) {
          F2 done[K];
          one(u, true, done);
          Pack<DT, V> p;
          pack_pairs(p, done);
          store_pack(to, p);
        }
      } else {
#pragma unroll 1
        for (int u = 0; u < U; ++u, to += P.ld_out) {
          const int tok = i + u;
          if (tok >= all_n) break;
          if (PACKED && tok >= q.hi) {
            flush(tok);
            if (tok >= n) {
              open = false;
              break;
            }
            q = conv_seq<PACKED>(P, batch, i0, tok);
            load_window<DT, V, W>(P, x, x0, q, tok, win);
            lo = group_lo(), hi = group_hi();
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
              for (int k = 0; k < K; ++k) wait[j][k] = 0;
          }
          F2 done[K];
          one(u, tok < n, done);
          emit(tok - (W - 1), done);
        }
      }
      ring.next();
      if ((i + U) % kSumTokens == 0) take_up();
    }
    if (open && i0 + all_n == P.s) flush(all_n);
    take_up();
  }
  if (P.ws == nullptr) return;

  // the block's parameter gradients: its slots in order
  cp_async_wait<0>();
  __syncthreads();                     // the rows' space is free
  float(*sums)[S + 1] = reinterpret_cast<float(*)[S + 1]>(space);
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float2 v = split(whole[j][k]);
      sums[threadIdx.x][2 * k * (W + 1) + j] = v.x;
      sums[threadIdx.x][(2 * k + 1) * (W + 1) + j] = v.y;
    }
    const float2 v = split(whole[W][k]);
    sums[threadIdx.x][2 * k * (W + 1) + W] = v.x;
    sums[threadIdx.x][(2 * k + 1) * (W + 1) + W] = v.y;
  }
  __syncthreads();
  const int first = (slab - r * per_rank) * P.lanes;
  const int live = P.vecs - first < P.lanes ? P.vecs - first : P.lanes;
  float* ws = P.ws + (static_cast<int64_t>(part) * P.t * P.c + static_cast<int64_t>(r) * P.c +
                      first * V) * (W + 1);
  for (int i = threadIdx.x; i < live * S; i += kConvThreads) {
    const int l = i / S, e = i - l * S;
    float a = 0.f;
    for (int k = 0; k < slots; ++k) a += sums[k * P.lanes + l][e];
    ws[i] = a;
  }
}

// dweight and dbias from the blocks' parts.
__global__ void __launch_bounds__(kPartThreads)
conv_params_kernel(const float* ws, int64_t channels, int width, int parts, float* dweight,
                   float* dbias) {
  pdl_wait();
  const int64_t n = channels * (width + 1);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
  const float a = sum_parts(ws, n, parts, i);
  if (threadIdx.x >= 32 || i >= n) return;
  const int64_t ch = i / (width + 1);
  const int j = static_cast<int>(i - ch * (width + 1));
  if (j < width) {
    if (dweight != nullptr) dweight[ch * width + j] = a;
  } else if (dbias != nullptr) {
    dbias[ch] = a;
  }
}

// The gradients of the states of packed sequences without a token pass.
template <int DT, int W>
__global__ void __launch_bounds__(kConvThreads)
conv_empty_kernel(const ConvParams P) {
  constexpr int V = kConvVec, E = ElemSize<DT>::value;
  pdl_wait();
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x;
  const int64_t slot = id / P.vecs;
  const int vec = static_cast<int>(id - slot * P.vecs);
  const int64_t r = slot / P.n_seqs;
  if (r >= P.t) return;
  const int64_t j = slot - r * P.n_seqs;
  if (__ldg(P.cu_seqlens + j) != __ldg(P.cu_seqlens + j + 1)) return;
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int64_t at = (j * (W - 1) + k) * P.c * E + vec * V * E;
    Pack<DT, V> p{};
    if (P.dxT[r] != nullptr) load_pack(p, P.dxT[r] + at);
    store_pack(P.xT[r] + at, p);
  }
}

template <int DT, int W>
static cudaError_t launch_width(ConvParams& p, cudaStream_t st) {
  void* args[] = {&p};
  const bool packed = p.cu_seqlens != nullptr;
  const void* fn = packed ? reinterpret_cast<const void*>(&conv_bwd_kernel<DT, W, true>)
                          : reinterpret_cast<const void*>(&conv_bwd_kernel<DT, W, false>);
  const cudaError_t e = launch_pdl(fn, dim3(static_cast<unsigned>(p.parts) * p.slabs),
                                   dim3(kConvThreads), 0, args, st);
  if (e != cudaSuccess || !packed || p.xT[0] == nullptr) return e;
  const int64_t rows = static_cast<int64_t>(p.n_seqs) * p.t * p.vecs;
  return launch_pdl(reinterpret_cast<const void*>(&conv_empty_kernel<DT, W>),
                    dim3(static_cast<unsigned>((rows + kConvThreads - 1) / kConvThreads)),
                    dim3(kConvThreads), 0, args, st);
}

template <int DT>
static cudaError_t launch_dtype(ConvParams& p, cudaStream_t st) {
  switch (p.width) {
    case 2: return launch_width<DT, 2>(p, st);
    case 3: return launch_width<DT, 3>(p, st);
    default: return launch_width<DT, 4>(p, st);
  }
}

// Vectors side by side in a block, its slabs, parts and runs.
static void conv_bwd_split(ConvParams* p, int64_t b, int64_t s, int c, int t) {
  p->vecs = c / kConvVec;
  // As many lanes side by side as leave fewer of them without a vector than half of those
  // that have one (2 x 3 x 1501 x 264, 66 vectors in 96 lanes 16.6 us, in 72 of them 17.2).
  p->lanes = 32;
  auto idle = [&] { return (p->lanes - p->vecs % p->lanes) % p->lanes; };
  while (p->lanes > 8 && idle() * 2 > p->vecs) p->lanes /= 2;
  p->slabs = t * ((p->vecs + p->lanes - 1) / p->lanes);
  const int64_t slots = kConvThreads / p->lanes, tokens = b * s;
  // One wave of blocks, whose threads have runs of 256 tokens or more, all as many.  (Every
  // run reads W - 1 rows twice and starts anew: 8 ranks' 16,384 x 1024, both directions,
  // 253 us with runs of 64 tokens, 239 of 128, 235 of 256 and of 512.)
  const int64_t wave = static_cast<int64_t>(device_sm_count()) * kConvBlocksB;
  int64_t parts = wave / p->slabs > 1 ? wave / p->slabs : 1;
  const int64_t least = (tokens + 4 * slots - 1) / (4 * slots);
  if (parts > least) parts = least;
  int64_t rounds = tokens / (slots * parts * 256);
  if (rounds < 1) rounds = 1;
  const int64_t pieces = slots * parts * rounds / b;             // of a batch row
  int64_t run = pieces > 1 ? (s + pieces - 1) / pieces : s;
  run = run < 4 ? 4 : run > 1024 ? 1024 : (run + 3) / 4 * 4;
  p->run = static_cast<int32_t>(run);
  p->runs = (s + run - 1) / run;
  const int64_t most = (p->runs * b + slots - 1) / slots;
  p->parts = static_cast<int32_t>(parts < most ? parts : most);
}

int conv_bwd_parts(int64_t b, int64_t s, int c, int t, int dtype) {
  ConvParams p{};
  conv_bwd_split(&p, b, s, c, t);
  return p.parts;
}

cudaError_t launch_conv_bwd(ConvParams p, int dtype, float* dweight, float* dbias,
                            cudaStream_t st) {
  conv_bwd_split(&p, p.b, p.s, p.c, p.t);
  cudaError_t e = dtype == SP_BF16  ? launch_dtype<SP_BF16>(p, st)
                  : dtype == SP_F16 ? launch_dtype<SP_F16>(p, st)
                                    : launch_dtype<SP_F32>(p, st);
  if (e != cudaSuccess || p.ws == nullptr) return e;
  int64_t channels = static_cast<int64_t>(p.t) * p.c;
  const float* ws = p.ws;
  void* args[] = {&ws, &channels, &p.width, &p.parts, &dweight, &dbias};
  const int64_t n = channels * (p.width + 1);
  return launch_pdl(reinterpret_cast<const void*>(&conv_params_kernel),
                    dim3(static_cast<unsigned>((n + 31) / 32)), dim3(kPartThreads), 0, args, st);
}

}  // namespace spb
