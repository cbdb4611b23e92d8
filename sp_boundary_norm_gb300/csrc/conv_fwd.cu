// Causal convolution, forward.  A thread takes four channels and a run of tokens, with
// the last W - 1 inputs in registers, so that each input is read once but for the W - 1
// rows before a run.  Rows on their way wait in shared memory (RowRing).  Bound by reading
// x and writing y: on a GB300, bf16, 8 ranks' packed 16,384 x 1024 with four taps and silu,
// 538 MB in 89 us, 6.0 TB/s (a copy reaches 6.8).  Rows asked for in registers took 110 us,
// a check of every row for its sequence's end 107, eight channels a thread 146.
#include "conv.cuh"

namespace spb {

template <int DT, int W, bool PACKED>
__global__ void __launch_bounds__(kConvThreads, 6)
conv_fwd_kernel(const ConvParams P) {
  constexpr int V = kConvVec, K = V / 2, E = ElemSize<DT>::value, U = kConvGroup;
  __shared__ __align__(16) char ring_space[RowRing<DT, V, 1>::kSize];
  pdl_wait();
  if (PACKED && blockIdx.x == 0 && threadIdx.x < 32)
    check_cu_seqlens(P.cu_seqlens, P.n_seqs, P.s, P.status);
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x;
  const int64_t most = P.runs * P.b * P.vecs * P.t;
  if (id >= most) return;
  const int64_t slot = divide(id, P.vecs, most);
  const int vec = static_cast<int>(id - slot * P.vecs);
  const int64_t row = divide(slot, P.runs, most), run = slot - row * P.runs;
  const int r = static_cast<int>(divide(row, P.b, most));
  const int64_t batch = row - static_cast<int64_t>(r) * P.b;
  const int64_t i0 = run * P.run;
  const int n = i0 + P.run < P.s ? P.run : static_cast<int>(P.s - i0);
  const char* x = P.x[r] + (batch * P.s + i0) * P.ld_x + vec * V * E;
  char* y = P.out[r] + (batch * P.s + i0) * P.ld_out + vec * V * E;
  const char* x0 = P.x0[r] != nullptr ? P.x0[r] + vec * V * E : nullptr;
  RowRing<DT, V, 1> ring(ring_space);
  ring.src[0] = x;
  ring.ld[0] = P.ld_x;
#pragma unroll
  for (int g = 0; g < kConvAhead; ++g) ring.ask(n - g * U);
  ConvSeq q = conv_seq<PACKED>(P, batch, i0, 0);
  F2 win[W - 1][K];
  load_window<DT, V, W>(P, x, x0, q, 0, win);
  Taps<DT, V, W> taps;
  taps.load(P, static_cast<int64_t>(r) * P.c + vec * V);
  auto one = [&](int u, char* dst) {
    Pack<DT, V> p;
    F2 v[K], o[K];
    ring.row(u, 0, p);
    unpack_pairs(p, v);
    taps.apply(win, v, o);
    shift<W, K>(win, v);
    if (P.act == SP_ACT_SILU) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        o[k] = mul2(o[k], rcp2(add2(exp2_of<DT, false, -1>(o[k]), f2(1.f, 1.f))));
    }
    pack_pairs(p, o);
    store_pack(dst, p);
  };
  for (int i = 0; i < n; i += U) {
    ring.ask(n - i - kConvAhead * U);
    cp_async_wait<kConvAhead>();
    if (i + U <= n && (!PACKED || i + U <= q.hi)) {
#pragma unroll
      for (int u = 0; u < U; ++u, y += P.ld_out) one(u, y);
    } else {                           // the run's end, or a sequence's
#pragma unroll 1
      for (int u = 0; u < U && i + u < n; ++u, y += P.ld_out) {
        if (PACKED && i + u >= q.hi) {
          q = conv_seq<PACKED>(P, batch, i0, i + u);
          load_window<DT, V, W>(P, x, x0, q, i + u, win);
        }
        one(u, y);
      }
    }
    ring.next();
  }
  // The state after a dense sequence comes from the thread of its first run, the only
  // one that reads x0 (a run has W - 1 tokens at least, or the whole sequence), so xT
  // may be x0.
  if (!PACKED && i0 == 0 && P.xT[r] != nullptr) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      Pack<DT, V> p;
      if (n == P.s) pack_pairs(p, win[j]);
      else load_pack(p, x + (P.s - (W - 1) + j) * P.ld_x);
      store_pack(P.xT[r] + (batch * (W - 1) + j) * P.c * E + vec * V * E, p);
    }
  }
}

// The states after packed sequences, when the forward is done with those before: a
// thread takes a sequence's vector of channels, reads its W - 1 rows and writes them.
template <int DT, int W>
__global__ void __launch_bounds__(kConvThreads)
conv_state_kernel(const ConvParams P) {
  constexpr int V = kConvVec, E = ElemSize<DT>::value;
  pdl_wait();
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x;
  const int64_t slot = id / P.vecs;
  const int vec = static_cast<int>(id - slot * P.vecs);
  const int64_t r = slot / P.n_seqs;
  if (r >= P.t) return;
  const int64_t j = slot - r * P.n_seqs;
  int64_t lo = __ldg(P.cu_seqlens + j), hi = __ldg(P.cu_seqlens + j + 1);
  lo = lo < 0 ? 0 : lo > P.s ? P.s : lo;            // in bounds whatever cu holds
  hi = hi < lo ? lo : hi > P.s ? P.s : hi;
  Pack<DT, V> rows[W - 1];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int64_t row = hi - (W - 1) + k;
    rows[k] = Pack<DT, V>{};
    if (row >= lo) load_pack(rows[k], P.x[r] + row * P.ld_x + vec * V * E);
    else if (P.x0[r] != nullptr)
      load_pack(rows[k], P.x0[r] + (j * (W - 1) + (W - 1 + row - lo)) * P.c * E + vec * V * E);
  }
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    store_pack(P.xT[r] + (j * (W - 1) + k) * P.c * E + vec * V * E, rows[k]);
}

template <int DT, int W>
static cudaError_t launch_width(ConvParams& p, cudaStream_t st) {
  const int64_t threads = p.runs * p.b * p.t * p.vecs;
  const unsigned grid = static_cast<unsigned>((threads + kConvThreads - 1) / kConvThreads);
  void* args[] = {&p};
  const bool packed = p.cu_seqlens != nullptr;
  const void* fn = packed ? reinterpret_cast<const void*>(&conv_fwd_kernel<DT, W, true>)
                          : reinterpret_cast<const void*>(&conv_fwd_kernel<DT, W, false>);
  const cudaError_t e = launch_pdl(fn, dim3(grid), dim3(kConvThreads), 0, args, st);
  if (e != cudaSuccess || !packed || p.xT[0] == nullptr) return e;
  const int64_t rows = static_cast<int64_t>(p.n_seqs) * p.t * p.vecs;
  return launch_pdl(reinterpret_cast<const void*>(&conv_state_kernel<DT, W>),
                    dim3(static_cast<unsigned>((rows + kConvThreads - 1) / kConvThreads)),
                    dim3(kConvThreads), 0, args, st);
}

template <int DT>
static cudaError_t launch_dtype(ConvParams& p, cudaStream_t st) {
  p.vecs = p.c / kConvVec;
  // runs of 64 tokens, or shorter ones until every SM has its warps
  const int64_t want = static_cast<int64_t>(device_sm_count()) * 1024;
  p.run = 64;
  while (p.run > 4 && (p.s + p.run - 1) / p.run * p.b * p.t * p.vecs < want) p.run /= 2;
  p.runs = (p.s + p.run - 1) / p.run;
  switch (p.width) {
    case 2: return launch_width<DT, 2>(p, st);
    case 3: return launch_width<DT, 3>(p, st);
    default: return launch_width<DT, 4>(p, st);
  }
}

cudaError_t launch_conv_fwd(ConvParams p, int dtype, cudaStream_t st) {
  return dtype == SP_BF16  ? launch_dtype<SP_BF16>(p, st)
         : dtype == SP_F16 ? launch_dtype<SP_F16>(p, st)
                           : launch_dtype<SP_F32>(p, st);
}

}  // namespace spb
