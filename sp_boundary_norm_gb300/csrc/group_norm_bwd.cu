// Group norm with an activation, backward.  With z and q recomputed from the
// saved statistics, dq = dy act'(q) and dz = dq gamma:
//   dx = rstd (dz - mean_group(dz) [LayerNorm] - z mean_group(dz z))
//   dgamma = sum over samples and rows of dq z,   dbeta = sum of dq
// A thread's column stays the same, so it sums its channels' dq z and dq in
// registers; each block writes one part of them and a second kernel adds the
// parts in order.  For a whole sample the group sums follow from the same
// channel sums: sum dz = sum_c gamma_c (sum dq), and so for dz z.
#include "group_norm.cuh"

namespace spb {


// z and dq in place of a vector's x and dy, its parts of the column's parameter
// gradients added to acc; its sums of dz and of dz z.
template <int DT>
__device__ __forceinline__ void back_vector(F2 (&z)[4], F2 (&dq)[4], float mean, float rstd,
                                            const Column<DT>& col, bool silu, F2 (&acc)[8],
                                            float& sum1, float& sum2) {
  back_act<DT>(z, dq, mean, rstd, col, silu);
  F2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[i] = fma2(dq[i], z[i], acc[i]);
    acc[4 + i] = add2(acc[4 + i], dq[i]);
    const F2 dz = mul2(dq[i], col.gamma[i]);
    s1 = add2(s1, dz);
    s2 = fma2(dz, z[i], s2);
  }
  const float2 w1 = split(s1), w2 = split(s2);
  sum1 = w1.x + w1.y;
  sum2 = w2.x + w2.y;
}

// Rows (as in the forward).
template <int DT, int MODE>
__global__ void __launch_bounds__(MODE == kSumTeam ? kGroupThreads : 32 * kRowWarps,
                                  MODE == kSumTeam ? 1 : kBackRowBlocks)
group_row_bwd_kernel(const GroupNormParams P) {
  constexpr int E = ElemSize<DT>::value;
  extern __shared__ float2 dyn2[];             // the parameter gradients' parts
  __shared__ RowSums<MODE, 2 * kBackRowRows> sh;
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team_warps = MODE == kSumTeam ? (P.cols + 31) / 32 : 1;
  const int team = warp / team_warps, cx = (warp - team * team_warps) * 32 + lane;
  const int slab = blockIdx.x % P.slabs;
  const int r = blockIdx.x / P.slabs % P.t;
  const int part = static_cast<int>(blockIdx.x) / (P.slabs * P.t);
  const int vec = slab * P.cols + cx;
  const bool on = cx < P.cols && vec * 8 < P.c;
  const bool ln = P.norm == SP_NORM_LAYERNORM, silu = P.act == SP_ACT_SILU;
  const int in_slab = cx < P.cols ? cx / P.q : 0;
  RowGroup<MODE, 2 * kBackRowRows> group{&sh, P.q, warp, in_slab * P.q, team_warps, team};
  const int64_t ch0 = static_cast<int64_t>(r) * P.c + slab * P.cols * 8, ch = ch0 + cx * 8;
  Column<DT> col;
  col.read(P, ch, on);
  const int64_t at = static_cast<int64_t>(vec) * 8 * E;
  const int64_t first = (static_cast<int64_t>(part) * P.rows + team) * kBackRowRows;
  const int64_t step = P.parts * P.rows * kBackRowRows;
  const char* x = P.x[r] + first * P.ld_x + at;
  const char* dy = P.dy[r] + first * P.ld_dy + at;
  char* out = P.out[r] + first * P.ld_out + at;
  const float* mean_at = ln ? P.mean[r] + first * P.groups + vec / P.q : nullptr;
  const float* rstd_at = P.rstd[r] + first * P.groups + vec / P.q;
  const int64_t step_x = step * P.ld_x, step_dy = step * P.ld_dy, step_out = step * P.ld_out;
  const int64_t step_stat = step * P.groups;
  F2 acc[8];                                   // dgamma, dbeta of the column
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = both(0.f);

  Vec8<DT> xraw[kBackRowRows], draw[kBackRowRows];
  float mean_next[kBackRowRows], rstd_next[kBackRowRows];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int u = 0; u < kBackRowRows; ++u) {
      xraw[u] = draw[u] = Vec8<DT>{};
      mean_next[u] = rstd_next[u] = 0.f;
      if (on && row + u < P.n) {
        load_pack(xraw[u], x + u * P.ld_x);
        load_pack(draw[u], dy + u * P.ld_dy);
        if (ln) mean_next[u] = __ldg(mean_at + u * P.groups);
        rstd_next[u] = __ldg(rstd_at + u * P.groups);
      }
    }
    x += step_x;
    dy += step_dy;
    if (ln) mean_at += step_stat;
    rstd_at += step_stat;
  };
  fetch(first);
  for (int64_t row = first; row < P.n; row += step, out += step_out) {
    F2 z[kBackRowRows][4], dq[kBackRowRows][4];
    float rstd[kBackRowRows];
    float sum[2 * kBackRowRows];              // of dz and of dz z
#pragma unroll
    for (int u = 0; u < kBackRowRows; ++u) {
      unpack_pairs(xraw[u], z[u]);
      unpack_pairs(draw[u], dq[u]);
      rstd[u] = rstd_next[u];
      back_vector<DT>(z[u], dq[u], mean_next[u], rstd[u], col, silu, acc, sum[2 * u],
                      sum[2 * u + 1]);
    }
    fetch(row + step);
    group.sum(sum);
#pragma unroll
    for (int u = 0; u < kBackRowRows; ++u) {
      if (!on || row + u >= P.n) continue;
      const float m1 = ln ? sum[2 * u] * P.count_inv : 0.f, m2 = sum[2 * u + 1] * P.count_inv;
      store_pack(out + u * P.ld_out, back_out<DT>(z[u], dq[u], rstd[u], col, m1, m2));
    }
  }
  if (P.has_params)
    put_param_part(P, acc, reinterpret_cast<float*>(dyn2), cx, on ? team : P.rows, ch0,
                   P.c - slab * P.cols * 8, part);
}

// Tiles: samples of a few rows.
template <int DT>
__global__ void __launch_bounds__(kGroupThreads) group_tile_bwd_kernel(const GroupNormParams P) {
  constexpr int E = ElemSize<DT>::value;
  extern __shared__ float2 dyn2[];             // [tile rows][cols] sums, then [pairs]
  pdl_wait();
  const int cx = threadIdx.x % P.cols, ry = threadIdx.x / P.cols;
  const int slab = blockIdx.x % P.slabs;
  const int r = blockIdx.x / P.slabs % P.t;
  const int part = static_cast<int>(blockIdx.x) / (P.slabs * P.t);
  const int vec = slab * P.cols + cx;
  const bool on = ry < P.rows && vec * 8 < P.c;
  const bool ln = P.norm == SP_NORM_LAYERNORM, silu = P.act == SP_ACT_SILU;
  const int64_t ch0 = static_cast<int64_t>(r) * P.c + slab * P.cols * 8, ch = ch0 + cx * 8;
  Column<DT> col;
  col.read(P, ch, on);
  const int64_t at = static_cast<int64_t>(vec) * 8 * E;
  const char* x = P.x[r] + at;
  const char* dy = P.dy[r] + at;
  char* out = P.out[r] + at;
  const int l = static_cast<int>(P.l), tile_rows = P.samples * l;
  const int slab_groups = P.cols / P.q;
  const int pairs = P.samples * slab_groups;
  float2* stat = dyn2 + P.rows * kBackTileRows * P.cols;
  const int group = vec / P.q;
  const int64_t all_rows = P.n * P.l, step = P.parts * P.samples;
  int pair[kBackTileRows], sample[kBackTileRows];
#pragma unroll
  for (int u = 0; u < kBackTileRows; ++u) {
    const int row = ry + u * P.rows;
    sample[u] = row / l;
    pair[u] = row < tile_rows ? sample[u] * slab_groups + cx / P.q : 0;
  }
  F2 acc[8];                                   // dgamma, dbeta of the column
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = both(0.f);

  Vec8<DT> xraw[kBackTileRows], draw[kBackTileRows];
  float mean_next[kBackTileRows], rstd_next[kBackTileRows];
  auto fetch = [&](int64_t s0) {
    const int64_t row0 = s0 * P.l, left = all_rows - row0;
    const int here = left < tile_rows ? static_cast<int>(left < 0 ? 0 : left) : tile_rows;
#pragma unroll
    for (int u = 0; u < kBackTileRows; ++u) {
      xraw[u] = draw[u] = Vec8<DT>{};
      mean_next[u] = rstd_next[u] = 0.f;
      const int row = ry + u * P.rows;
      if (on && row < here) {
        load_pack(xraw[u], x + (row0 + row) * P.ld_x);
        load_pack(draw[u], dy + (row0 + row) * P.ld_dy);
        const int64_t st = (s0 + sample[u]) * P.groups + group;
        if (ln) mean_next[u] = __ldg(P.mean[r] + st);
        rstd_next[u] = __ldg(P.rstd[r] + st);
      }
    }
  };
  const int64_t s_first = static_cast<int64_t>(part) * P.samples;
  fetch(s_first);
  for (int64_t s0 = s_first; s0 < P.n; s0 += step) {
    const int64_t row0 = s0 * P.l;
    const int64_t left = all_rows - row0;
    const int here = left < tile_rows ? static_cast<int>(left) : tile_rows;
    F2 z[kBackTileRows][4], dq[kBackTileRows][4];
    float rstd[kBackTileRows];
#pragma unroll
    for (int u = 0; u < kBackTileRows; ++u) {
      unpack_pairs(xraw[u], z[u]);
      unpack_pairs(draw[u], dq[u]);
      rstd[u] = rstd_next[u];
      float2 sum;
      back_vector<DT>(z[u], dq[u], mean_next[u], rstd[u], col, silu, acc, sum.x, sum.y);
      if (ry < P.rows) dyn2[(ry + u * P.rows) * P.cols + cx] = sum;
    }
    fetch(s0 + step);
    __syncthreads();
    const int lane = threadIdx.x % P.lanes, teams = blockDim.x / P.lanes;
    for (int p0 = 0; p0 < pairs; p0 += teams) {
      const int p = p0 + threadIdx.x / P.lanes;
      float v[2] = {0.f, 0.f};
      if (p < pairs) {
        const int s = p / slab_groups;
        const float2* from = dyn2 + s * l * P.cols + (p - s * slab_groups) * P.q;
        for (int i = 0; i < l; ++i, from += P.cols)
          for (int j = lane; j < P.q; j += P.lanes) {
            v[0] += from[j].x;
            v[1] += from[j].y;
          }
      }
      lanes_sum(v, P.lanes);
      if (p < pairs && lane == 0) stat[p] = make_float2(v[0], v[1]);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kBackTileRows; ++u) {
      const int row = ry + u * P.rows;
      if (!on || row >= here) continue;
      const float2 w = stat[pair[u]];
      const float m1 = ln ? w.x * P.count_inv : 0.f, m2 = w.y * P.count_inv;
      store_pack(out + (row0 + row) * P.ld_out,
                 back_out<DT>(z[u], dq[u], rstd[u], col, m1, m2));
    }
    __syncthreads();                           // the next tile's sums replace these
  }
  if (P.has_params)
    put_param_part(P, acc, reinterpret_cast<float*>(dyn2), cx, ry, ch0, P.c - slab * P.cols * 8,
                   part);
}

// A cluster's group means of dz and dz z of its sample's slab from `sums`, those
// of each thread's values.
__device__ __forceinline__ void join_sums(const GroupNormParams& P, int C, int rank,
                                          const float2* sums, float2* joined, float2* stat) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int slab_groups = P.cols / P.q;
  const bool ln = P.norm == SP_NORM_LAYERNORM;
  __syncthreads();
  if (C > 1) cluster_wait();                   // the partners run: their shared memory is there
  for (int g = warp; g < slab_groups; g += nw) {
    float2 v = make_float2(0.f, 0.f);
    group_entries(P, g, [&](int, int at) {
      v.x += sums[at].x;
      v.y += sums[at].y;
    });
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if (C == 1) {
      if (lane == 0) stat[g] = make_float2(ln ? v.x * P.count_inv : 0.f, v.y * P.count_inv);
    } else if (lane < C) {
      const uint32_t to = cluster_map(&joined[rank * slab_groups + g], lane);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(v.x), "f"(v.y)
                   : "memory");
    }
  }
  if (C > 1) {
    cluster_sync_all();
    for (int g = threadIdx.x; g < slab_groups; g += blockDim.x) {
      float2 v = make_float2(0.f, 0.f);
      for (int k = 0; k < C; ++k) {
        v.x += joined[k * slab_groups + g].x;
        v.y += joined[k * slab_groups + g].y;
      }
      stat[g] = make_float2(ln ? v.x * P.count_inv : 0.f, v.y * P.count_inv);
    }
  }
  __syncthreads();
}

// Held (as in the forward).
template <int DT>
__global__ void __launch_bounds__(256, kHeldBlocks) group_held_bwd_kernel(const GroupNormParams P) {
  constexpr int E = ElemSize<DT>::value, kMost = kBackHold<DT>;
  extern __shared__ float2 sums[];             // [threads] sums of dz and dz z
  pdl_wait();
  const int cx = threadIdx.x % P.cols, ry = threadIdx.x / P.cols;
  const int slab = blockIdx.x % P.slabs;
  const int r = blockIdx.x / P.slabs % P.t;
  const int part = static_cast<int>(blockIdx.x) / (P.slabs * P.t);
  const int vec = slab * P.cols + cx;
  const bool on = ry < P.rows && vec * 8 < P.c;
  const bool ln = P.norm == SP_NORM_LAYERNORM, silu = P.act == SP_ACT_SILU;
  float2* stat = sums + blockDim.x;            // [slab groups] group means of dz and dz z
  const int64_t ch0 = static_cast<int64_t>(r) * P.c + slab * P.cols * 8, ch = ch0 + cx * 8;
  const Deal lanes(static_cast<int>(P.l), P.rows);
  const int mine = on ? lanes.count(ry) : 0;
  const int64_t row0 = part * P.l + ry;
  const int64_t at = static_cast<int64_t>(vec) * 8 * E;
  const char* x = P.x[r] + row0 * P.ld_x + at;
  const char* dy = P.dy[r] + row0 * P.ld_dy + at;
  char* out = P.out[r] + row0 * P.ld_out + at;
  const int64_t step_x = P.ld_x * P.rows, step_dy = P.ld_dy * P.rows, step_out = P.ld_out * P.rows;
  const int64_t skip = P.parts * P.l;          // rows from sample to sample
  Column<DT> col;
  col.read(P, ch, on);
  F2 acc[8];                                   // dgamma, dbeta of the column
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = both(0.f);
  for (int64_t sample = part; sample < P.n; sample += P.parts) {
    Vec8<DT> xraw[kMost], draw[kMost];
    const char *from = x, *dfrom = dy;
#pragma unroll
    for (int u = 0; u < kMost; ++u, from += step_x, dfrom += step_dy)
      if (u < mine) {
        load_pack(xraw[u], from);
        load_pack(draw[u], dfrom);
      }
    float mean = 0.f, rstd = 0.f;
    if (on) {
      const int64_t g = sample * P.groups + vec / P.q;
      if (ln) mean = __ldg(P.mean[r] + g);
      rstd = __ldg(P.rstd[r] + g);
    }
    F2 z[4], dq[4];
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < kMost; ++u)
      if (u < mine) {
        unpack_pairs(xraw[u], z);
        unpack_pairs(draw[u], dq);
        float s1, s2;
        back_vector<DT>(z, dq, mean, rstd, col, silu, acc, s1, s2);
        sum.x += s1;
        sum.y += s2;
      }
    if (ry < P.rows) sums[threadIdx.x] = sum;
    join_sums(P, 1, 0, sums, nullptr, stat);
    const float2 m = stat[on ? cx / P.q : 0];
    char* to = out;
#pragma unroll
    for (int u = 0; u < kMost; ++u, to += step_out)
      if (u < mine) {
        unpack_pairs(xraw[u], z);
        unpack_pairs(draw[u], dq);
        back_act<DT>(z, dq, mean, rstd, col, silu);
        store_pack(to, back_out<DT>(z, dq, rstd, col, m.x, m.y));
      }
    x += skip * P.ld_x;
    dy += skip * P.ld_dy;
    out += skip * P.ld_out;
  }
  if (P.has_params)
    put_param_part(P, acc, reinterpret_cast<float*>(sums), cx, ry, ch0, P.c - slab * P.cols * 8,
                   part);
}

template <int DT, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kGroupThreads : 256, WIDE ? 1 : kBackUnitBlocks)
group_unit_bwd_kernel(const GroupNormParams P) {
  constexpr int E = ElemSize<DT>::value, kRing = kBackUnitRing<DT>;
  extern __shared__ float2 sums[];             // [threads] sums of dz and dz z
  const int C = P.cluster, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  if (C > 1) cluster_arrive();                 // waited for before the first remote store
  pdl_wait();
  const int cx = threadIdx.x % P.cols, ry = threadIdx.x / P.cols;
  int unit = static_cast<int>(blockIdx.x) / C;
  const int slab = unit % P.slabs;
  unit /= P.slabs;
  const int r = unit % P.t;
  const int sample = unit / P.t;
  const int vec = slab * P.cols + cx;
  const bool on = ry < P.rows && vec * 8 < P.c;
  const bool ln = P.norm == SP_NORM_LAYERNORM, silu = P.act == SP_ACT_SILU;
  float2* joined = sums + blockDim.x;          // [cluster][slab groups] sums of each block
  float2* stat = joined + C * (P.cols / P.q);  // [slab groups] group means of dz and dz z
  const int64_t ch0 = static_cast<int64_t>(r) * P.c + slab * P.cols * 8, ch = ch0 + cx * 8;
  const Deal blocks(static_cast<int>(P.l), C);
  const int b0 = blocks.first(rank), block_rows = blocks.count(rank);
  const Deal lanes(block_rows, P.rows);
  const int mine = on ? lanes.count(ry) : 0;
  const int64_t row0 = sample * P.l + b0 + ry;
  const int64_t at = static_cast<int64_t>(vec) * 8 * E;
  const char* x = P.x[r] + row0 * P.ld_x + at;
  const char* dy = P.dy[r] + row0 * P.ld_dy + at;
  char* out = P.out[r] + row0 * P.ld_out + at;
  const int64_t step_x = P.ld_x * P.rows, step_dy = P.ld_dy * P.rows, step_out = P.ld_out * P.rows;
  Column<DT> col;
  col.read(P, ch, on);
  float mean = 0.f, rstd = 0.f;
  if (on) {
    const int64_t g = sample * P.groups + vec / P.q;
    if (ln) mean = __ldg(P.mean[r] + g);
    rstd = __ldg(P.rstd[r] + g);
  }
  F2 acc[8];                                   // dgamma, dbeta of the column
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = both(0.f);
  // a vector's place is filled again as soon as it is used
  Vec8<DT> xraw[kRing], draw[kRing];
  const char *from = x, *dfrom = dy;
  auto fetch = [&](int u, int i, bool again) {
    if (i < mine) {
      if (again) {
        load_again<DT>(xraw[u], from);
        load_again<DT>(draw[u], dfrom);
      } else {
        load_pack(xraw[u], from);
        load_pack(draw[u], dfrom);
      }
    }
    from += step_x;
    dfrom += step_dy;
  };
  F2 z[4], dq[4];
#pragma unroll
  for (int u = 0; u < kRing; ++u) fetch(u, u, true);
  for (int i0 = 0; i0 < mine; i0 += kRing) {
#pragma unroll
    for (int u = 0; u < kRing; ++u) {
      unpack_pairs(xraw[u], z);
      unpack_pairs(draw[u], dq);
      fetch(u, i0 + kRing + u, true);
      if (i0 + u >= mine) continue;
      back_act<DT>(z, dq, mean, rstd, col, silu);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i] = fma2(dq[i], z[i], acc[i]);
        acc[4 + i] = add2(acc[4 + i], dq[i]);
      }
    }
  }
  from = x;
  dfrom = dy;
#pragma unroll
  for (int u = 0; u < kRing; ++u) fetch(u, u, false);
  F2 own1 = both(0.f), own2 = both(0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    own1 = fma2(col.gamma[i], acc[4 + i], own1);
    own2 = fma2(col.gamma[i], acc[i], own2);
  }
  const float2 w1 = split(own1), w2 = split(own2);
  if (ry < P.rows) sums[threadIdx.x] = make_float2(w1.x + w1.y, w2.x + w2.y);
  join_sums(P, C, rank, sums, joined, stat);
  const float2 m = stat[cx / P.q];
  for (int i0 = 0; i0 < mine; i0 += kRing) {
#pragma unroll
    for (int u = 0; u < kRing; ++u, out += step_out) {
      unpack_pairs(xraw[u], z);
      unpack_pairs(draw[u], dq);
      fetch(u, i0 + kRing + u, false);
      if (i0 + u >= mine) continue;
      back_act<DT>(z, dq, mean, rstd, col, silu);
      store_pack(out, back_out<DT>(z, dq, rstd, col, m.x, m.y));
    }
  }
  if (P.has_params)
    put_param_part(P, acc, reinterpret_cast<float*>(sums), cx, ry, ch0, P.c - slab * P.cols * 8,
                   static_cast<int64_t>(sample) * C + rank);
}

// dgamma / dbeta: the parts added in order, one warp lane a channel, eight
// partial sums of fixed strides per block of 32 channels.
__global__ void __launch_bounds__(256) group_params_kernel(const float* ws, int64_t parts,
                                                           int64_t width, float* dgamma,
                                                           float* dbeta) {
  __shared__ float sums[8][33];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t ch = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float* out = blockIdx.y == 0 ? dgamma : dbeta;
  float v = 0.f;
  if (out != nullptr && ch < width) {
    const float* src = ws + blockIdx.y * width + ch;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t k = warp; k < parts; k += 32) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k + 8 * u < parts) w[u] += __ldcs(src + (k + 8 * u) * 2 * width);
    }
    v = (w[0] + w[1]) + (w[2] + w[3]);
  }
  sums[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || out == nullptr || ch >= width) return;
  v = 0.f;
  for (int k = 0; k < 8; ++k) v += sums[k][lane];
  out[ch] = v;
}

template <int DT>
static const void* bwd_fn(const GroupShape& s) {
  if (s.form == kRowForm)
    return s.mode == kSumLanes  ? reinterpret_cast<const void*>(&group_row_bwd_kernel<DT, kSumLanes>)
           : s.mode == kSumWarp ? reinterpret_cast<const void*>(&group_row_bwd_kernel<DT, kSumWarp>)
                                : reinterpret_cast<const void*>(&group_row_bwd_kernel<DT, kSumTeam>);
  if (s.form == kTileForm) return reinterpret_cast<const void*>(&group_tile_bwd_kernel<DT>);
  if (s.form == kHeldForm) return reinterpret_cast<const void*>(&group_held_bwd_kernel<DT>);
  return s.threads > 256 ? reinterpret_cast<const void*>(&group_unit_bwd_kernel<DT, true>)
                         : reinterpret_cast<const void*>(&group_unit_bwd_kernel<DT, false>);
}

cudaError_t launch_group_norm_bwd(GroupNormParams p, int dtype, float* dgamma, float* dbeta,
                                  cudaStream_t st) {
  p.has_params = dgamma != nullptr || dbeta != nullptr;
  const GroupShape s = group_norm_shape(p.n, p.l, p.c, p.groups, p.t, dtype, true);
  const void* fn = dtype == SP_BF16  ? bwd_fn<SP_BF16>(s)
                   : dtype == SP_F16 ? bwd_fn<SP_F16>(s)
                                     : bwd_fn<SP_F32>(s);
  const cudaError_t e = launch_group(fn, &p, s, st);
  if (e != cudaSuccess || !p.has_params) return e;
  const float* ws = p.ws;
  int64_t parts = p.parts, width = static_cast<int64_t>(p.t) * p.c;
  void* args[] = {&ws, &parts, &width, &dgamma, &dbeta};
  return launch_pdl(reinterpret_cast<const void*>(&group_params_kernel),
                    dim3(static_cast<unsigned>((width + 31) / 32), 2), dim3(256), 0, args, st);
}

}  // namespace spb
