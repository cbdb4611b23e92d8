// Rotary positions: every rotated pair (u, v) of a head becomes
//   (m (u cos x - v sin x), m (v cos x + u sin x)),   x = position * frequency,
// and the backward is the same with -sin (the transpose of a rotation, times m).
//
// The angle is reduced exactly: a frequency is held as a 64-bit fraction of a
// turn, position * fraction mod 2^64 is the exact part of a turn however far
// the position (one wide integer multiply), its top 32 bits become a float in
// [-1, 1) half-turns for sincospif.
//
// One warp takes one token and a piece of its heads over all ranks: the lanes
// compute the token's sines and cosines once into shared memory, each lane
// keeps those of its own vector of pairs in registers and walks the heads, so
// a pair costs one rotation and its share of two loads and two stores.
// Bound by HBM: reads x once, writes y once.  Measured on a GB300, bf16, packed
// sequences of 16,384 tokens: 8 ranks of 9 heads of 128 95 us, 6.4 TB/s, 94 % of
// the measured copy rate (interleaved 96); 16 heads of 256 of which 64 turn 55;
// 64 tokens of 8 ranks' 8 heads 3.1, which is the launch and one trip to memory.
#include "region.cuh"

namespace spb {

constexpr int kRopeWarps = 8;
// Rounds of heads side by side that a lane reads at once; twice as many where an
// item is one 16-byte load (interleaved, 8 ranks of 9 heads of 128: 97 us, with
// four 101).
constexpr int kRopeRounds = 4;

// a / b for 0 <= a < most: in 32 bits where they do (a 64-bit division costs a
// hundred instructions).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b, int64_t most) {
  if (b == 1) return a;
  if (b >= most) return 0;
  if (most <= 0x7FFFFFFF) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

__device__ __forceinline__ int rank_of_head(const RopeParams& P, int hh) {
  return P.heads == 1 ? hh : static_cast<int>(__umulhi(static_cast<uint32_t>(hh), P.heads_magic));
}

// Blocks an SM that the registers are held to, by what a lane has on its way: two
// where an item is two 16-byte loads (half layout, 9 heads of 128 95 us, with four
// 100; 16 heads of 256 of which 64 turn 57 against 77), else four (5 heads of 80 of
// which 20 turn 26 us, with two 34).
constexpr int rope_blocks(int dt, int v, int layout) {
  const int bytes = v * (dt == SP_F32 ? 4 : 2) * (layout == SP_ROPE_HALF || v == 1 ? 2 : 1);
  return bytes >= 32 ? 2 : 4;
}

// What follows the rotated elements of a token's heads h0 .. h1 - 1 is copied B
// bytes a lane, several heads side by side and kRestRounds rounds at once; the
// first of them are asked for before the angles and wait in `held` (4 ranks, 8192
// tokens, 9 heads of 80 of which 20 turn: 24 us, asked for afterwards 27).
constexpr int kRestRounds = 4;
using Held = Pack<SP_BF16, 8>[kRestRounds];

template <int B, typename Use>
__device__ __forceinline__ void rest_rounds(const RopeParams& P, int hb, int h1, int abreast,
                                            int sub, Use use) {
#pragma unroll
  for (int k = 0; k < kRestRounds; ++k) {
    const int hh = hb + k * abreast + sub;
    if (sub < abreast && hh < h1) {
      const int r = rank_of_head(P, hh);
      use(k, r, hh - r * P.heads);
    }
  }
}

// PHASE 0: asks for the first; 1: stores them and copies the others.
template <int B, int PHASE>
__device__ __forceinline__ void copy_rest(const RopeParams& P, int64_t tok, int h0, int h1,
                                          Held& held) {
  using Piece = Pack<SP_BF16, B / 2>;
  const int lane = threadIdx.x & 31;
  const int items = P.rest / B, width = items < 32 ? items : 32, abreast = 32 / width;
  const int my = lane % width, sub = lane / width;
  const int64_t x_at = tok * P.x_row + P.rest_at, y_at = tok * P.y_row + P.rest_at;
  auto load = [&](int item, int hb) {
    rest_rounds<B>(P, hb, h1, abreast, sub, [&](int k, int r, int h) {
      Piece p;
      load_pack(p, P.x[r] + x_at + h * P.x_head + item * B);
#pragma unroll
      for (int i = 0; i < Piece::kWords; ++i) held[k].w[i] = p.w[i];
    });
  };
  if constexpr (PHASE == 0) {
    load(my, h0);
  } else {
    for (int item = my; item < items; item += width) {
      for (int hb = h0; hb < h1; hb += abreast * kRestRounds) {
        if (item != my || hb != h0) load(item, hb);
        rest_rounds<B>(P, hb, h1, abreast, sub, [&](int k, int r, int h) {
          Piece p;
#pragma unroll
          for (int i = 0; i < Piece::kWords; ++i) p.w[i] = held[k].w[i];
          store_pack(P.y[r] + y_at + h * P.y_head + item * B, p);
        });
      }
    }
  }
}
template <int PHASE>
__device__ __forceinline__ void copy_rest(const RopeParams& P, int64_t tok, int h0, int h1,
                                          Held& held) {
  if (P.rest == 0) return;
  if (P.rest_bytes == 16) copy_rest<16, PHASE>(P, tok, h0, h1, held);
  else if (P.rest_bytes == 8) copy_rest<8, PHASE>(P, tok, h0, h1, held);
  else if (P.rest_bytes == 4) copy_rest<4, PHASE>(P, tok, h0, h1, held);
  else copy_rest<2, PHASE>(P, tok, h0, h1, held);
}

// V elements a load.  Half layout: a lane's item is V pairs (V elements of
// each half).  Interleaved: V / 2 pairs that lie together, or for V = 1 one
// pair by two loads.
template <int DT, int V, int LAYOUT>
__global__ void __launch_bounds__(32 * kRopeWarps, rope_blocks(DT, V, LAYOUT))
rope_kernel(const RopeParams P) {
  constexpr int E = ElemSize<DT>::value;
  constexpr bool kTwo = LAYOUT == SP_ROPE_HALF || V == 1;   // an item is two loads
  constexpr int U = kTwo || V * E < 16 ? kRopeRounds : 2 * kRopeRounds;
  constexpr int kPairs = kTwo ? V : V / 2;
  __shared__ float2 cs[kRopeWarps][SP_ROPE_MAX_PAIRS];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && warp == 0)
    check_cu_seqlens(P.cu_seqlens, P.n_seqs, P.s, P.status);
  const int items = P.half / kPairs;                 // of a head
  const int width = items < 32 ? items : 32;         // lanes of a head
  const int abreast = 32 / width;                    // heads side by side
  const int my = lane % width, sub = lane / width;
  constexpr int kStep = (V == 1 && LAYOUT != SP_ROPE_HALF ? 2 : V) * E;   // bytes between items
  // bytes from an item's first load to its second
  const uint32_t second = LAYOUT == SP_ROPE_HALF ? static_cast<uint32_t>(P.half) * E : E;
  const int64_t n_tasks = P.tokens * P.chunks;
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp; task < n_tasks;
       task += static_cast<int64_t>(gridDim.x) * kRopeWarps) {
    const int64_t tok = divide(task, P.chunks, n_tasks);
    const int chunk = static_cast<int>(task - tok * P.chunks);
    const int h0 = chunk * P.chunk_heads;
    const int h1 = h0 + P.chunk_heads < P.all_heads ? h0 + P.chunk_heads : P.all_heads;
    Pack<DT, V> a[U], b[U];
    auto fetch = [&](int hb, int item) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int hh = hb + k * abreast + sub;
        if (sub < abreast && item < items && hh < h1) {
          const int r = rank_of_head(P, hh);
          const char* src = P.x[r] + tok * P.x_row + (hh - r * P.heads) * P.x_head + item * kStep;
          load_pack(a[k], src);
          if constexpr (kTwo) load_pack(b[k], src + second);
        }
      }
    };
    // the first heads are on their way while the angles are computed
    fetch(h0, my);
    Held held;
    copy_rest<0>(P, tok, h0, h1, held);
    int64_t pos;
    if (P.positions != nullptr) {
      pos = __ldg(P.positions + tok);
    } else if (P.cu_seqlens != nullptr) {
      pos = tok - __ldg(P.cu_seqlens + seq_of_token(P.cu_seqlens, P.n_seqs, tok)) + P.first;
    } else {
      pos = tok - divide(tok, P.s, P.tokens) * P.s + P.first;
    }
    __syncwarp();
    for (int i = lane; i < P.half; i += 32) {
      const uint64_t turn = static_cast<uint64_t>(pos) * P.turns[i];
      const float half_turns =
          static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
      float sn, cn;
      sincospif(half_turns, &sn, &cn);
      cs[warp][i] = make_float2(cn * P.cos_scale, sn * P.sin_scale);
    }
    __syncwarp();
    for (int v0 = 0; v0 < items; v0 += width) {
      const int item = v0 + my;
      const bool on = sub < abreast && item < items;
      float cn[kPairs], sn[kPairs];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 v = on ? cs[warp][item * kPairs + i] : make_float2(0.f, 0.f);
        cn[i] = v.x;
        sn[i] = v.y;
      }
      for (int hb = h0; hb < h1; hb += abreast * U) {
        if (v0 > 0 || hb > h0) fetch(hb, item);
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int hh = hb + k * abreast + sub;
          if (on && hh < h1) {
            const int r = rank_of_head(P, hh);
            char* dst = P.y[r] + tok * P.y_row + (hh - r * P.heads) * P.y_head + item * kStep;
            float x[V];
            unpack(a[k], x);
            if constexpr (kTwo) {
              float z[V];
              unpack(b[k], z);
#pragma unroll
              for (int i = 0; i < V; ++i) {
                const float u = x[i], w = z[i];
                x[i] = u * cn[i] - w * sn[i];
                z[i] = w * cn[i] + u * sn[i];
              }
              pack(a[k], x);
              pack(b[k], z);
              store_pack(dst, a[k]);
              store_pack(dst + second, b[k]);
            } else {
#pragma unroll
              for (int i = 0; i < kPairs; ++i) {
                const float u = x[2 * i], w = x[2 * i + 1];
                x[2 * i] = u * cn[i] - w * sn[i];
                x[2 * i + 1] = w * cn[i] + u * sn[i];
              }
              pack(a[k], x);
              store_pack(dst, a[k]);
            }
          }
        }
      }
    }
    copy_rest<1>(P, tok, h0, h1, held);
  }
}

template <int DT, int V>
static const void* rope_fn(int layout) {
  return layout == SP_ROPE_HALF ? reinterpret_cast<const void*>(&rope_kernel<DT, V, SP_ROPE_HALF>)
                                : reinterpret_cast<const void*>(
                                      &rope_kernel<DT, V, SP_ROPE_INTERLEAVED>);
}

template <int DT>
static const void* rope_fn(int layout, int vec) {
  switch (vec) {
    case 1: return rope_fn<DT, 1>(layout);
    case 2: return rope_fn<DT, 2>(layout);
    case 4: return rope_fn<DT, 4>(layout);
    default:
      if constexpr (DT == SP_F32) return nullptr;
      else return rope_fn<DT, 8>(layout);
  }
}

cudaError_t launch_rope(RopeParams p, int dtype, int vec, cudaStream_t st) {
  // One warp a token, or few tokens' heads cut into pieces of whole lane rounds
  // until every SM has the warps that it holds at once.  (More pieces make a second
  // wave: 4096 tokens of 9 heads of 128 7 us, cut until four times as many warps
  // 14; 2 x 5997 tokens of 5 heads of 80 7.7 us, twice as many 10.4.)
  const int pairs = vec == 1 || p.layout == SP_ROPE_HALF ? vec : vec / 2;
  const int items = p.half / pairs;
  const int abreast = 32 / (items < 32 ? items : 32);
  const int rounds = (p.all_heads + abreast - 1) / abreast;
  const int64_t want = static_cast<int64_t>(device_sm_count()) *
                       rope_blocks(dtype, vec, p.layout) * kRopeWarps;
  int64_t chunks = p.tokens < want ? (want + p.tokens - 1) / p.tokens : 1;
  if (chunks > rounds) chunks = rounds;
  p.chunk_heads = static_cast<int>((rounds + chunks - 1) / chunks) * abreast;
  p.chunks = (p.all_heads + p.chunk_heads - 1) / p.chunk_heads;
  const void* fn = dtype == SP_BF16  ? rope_fn<SP_BF16>(p.layout, vec)
                   : dtype == SP_F16 ? rope_fn<SP_F16>(p.layout, vec)
                                     : rope_fn<SP_F32>(p.layout, vec);
  if (fn == nullptr) return cudaErrorInvalidValue;
  const int64_t blocks = (p.tokens * p.chunks + kRopeWarps - 1) / kRopeWarps;
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 8;
  void* args[] = {&p};
  return launch_pdl(fn, dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)),
                    dim3(32 * kRopeWarps), 0, args, st);
}

}  // namespace spb
