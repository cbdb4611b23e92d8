// Group norm with an activation, forward (the forms are described in
// group_norm.cuh), and the split of a call over the GPU for both directions.
#include "group_norm.cuh"

namespace spb {

// Rows: a team takes kRowRows rows of its slab at a time; the next ones are on
// their way meanwhile.
template <int DT, int MODE>
__global__ void __launch_bounds__(MODE == kSumTeam ? kGroupThreads : 32 * kRowWarps,
                                  MODE == kSumTeam ? 1 : kRowBlocks<DT>)
group_row_fwd_kernel(const GroupNormParams P) {
  constexpr int E = ElemSize<DT>::value, kRows = kRowRows<DT>;
  __shared__ RowSums<MODE, kRows> sh;
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
  RowGroup<MODE, kRows> group{&sh, P.q, warp, in_slab * P.q, team_warps, team};
  Column<DT> col;
  col.read(P, static_cast<int64_t>(r) * P.c + vec * 8, on);
  const bool tells = on && cx == in_slab * P.q;          // writes its group's statistics
  const int64_t first = (static_cast<int64_t>(part) * P.rows + team) * kRows;
  const int64_t step = P.parts * P.rows * kRows;
  const char* x = P.x[r] + first * P.ld_x + static_cast<int64_t>(vec) * 8 * E;
  char* out = P.out[r] + first * P.ld_out + static_cast<int64_t>(vec) * 8 * E;
  const int64_t step_x = step * P.ld_x, step_out = step * P.ld_out, step_stat = step * P.groups;
  float* rstd_at = P.rstd[r] + first * P.groups + vec / P.q;
  float* mean_at = ln ? P.mean[r] + first * P.groups + vec / P.q : nullptr;

  Vec8<DT> raw[kRows];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      raw[u] = Vec8<DT>{};
      if (on && row + u < P.n) load_pack(raw[u], x + u * P.ld_x);
    }
    x += step_x;
  };
  fetch(first);
  for (int64_t row = first; row < P.n; row += step, out += step_out) {
    F2 v[kRows][4];
#pragma unroll
    for (int u = 0; u < kRows; ++u) unpack_pairs(raw[u], v[u]);
    fetch(row + step);
    float mean[kRows], rstd[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) mean[u] = 0.f;
    if (ln) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) mean[u] = pair_sum(v[u]);
      group.sum(mean);
#pragma unroll
      for (int u = 0; u < kRows; ++u) mean[u] = mean_of(mean[u], P.count, P.count_inv);
    }
    // (lanes that hold no vector hold zeros: they add nothing)
#pragma unroll
    for (int u = 0; u < kRows; ++u) rstd[u] = on ? spread_sum(v[u], mean[u]) : 0.f;
    group.sum(rstd);
#pragma unroll
    for (int u = 0; u < kRows; ++u) rstd[u] = rsqrtf(rstd[u] * P.count_inv + P.eps);
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (!on || row + u >= P.n) continue;
      store_pack(out + u * P.ld_out, norm_act<DT>(v[u], rstd[u], col, silu));
      if (tells) {
        rstd_at[u * P.groups] = rstd[u];
        if (ln) mean_at[u * P.groups] = mean[u];
      }
    }
    rstd_at += step_stat;
    if (ln) mean_at += step_stat;
  }
}

// Tiles: samples of a few rows, several a block; each thread's place in a tile
// stays the same, and the next tile is on its way meanwhile.
template <int DT>
__global__ void __launch_bounds__(kGroupThreads) group_tile_fwd_kernel(const GroupNormParams P) {
  constexpr int E = ElemSize<DT>::value;
  extern __shared__ float dyn[];               // [tile rows][cols] sums, then [pairs] statistics
  pdl_wait();
  const int cx = threadIdx.x % P.cols, ry = threadIdx.x / P.cols;
  const int slab = blockIdx.x % P.slabs;
  const int r = blockIdx.x / P.slabs % P.t;
  const int part = static_cast<int>(blockIdx.x) / (P.slabs * P.t);
  const int vec = slab * P.cols + cx;
  const bool on = ry < P.rows && vec * 8 < P.c;
  const bool ln = P.norm == SP_NORM_LAYERNORM, silu = P.act == SP_ACT_SILU;
  Column<DT> col;
  col.read(P, static_cast<int64_t>(r) * P.c + vec * 8, on);
  const char* x = P.x[r] + static_cast<int64_t>(vec) * 8 * E;
  char* out = P.out[r] + static_cast<int64_t>(vec) * 8 * E;
  const int l = static_cast<int>(P.l), tile_rows = P.samples * l;
  const int slab_groups = P.cols / P.q;
  const int pairs = P.samples * slab_groups;
  float* stat = dyn + P.rows * kTileRows * P.cols;     // mean then rstd of each pair
  const int group = vec / P.q;
  const int64_t all_rows = P.n * P.l, step = P.parts * P.samples;
  int pair[kTileRows];                         // of this thread's rows; 0 for none
  bool leads[kTileRows];                       // the first row and column of a pair
#pragma unroll
  for (int u = 0; u < kTileRows; ++u) {
    const int row = ry + u * P.rows, s = row / l;
    pair[u] = row < tile_rows ? s * slab_groups + cx / P.q : 0;
    leads[u] = vec % P.q == 0 && row == s * l;
  }

  Vec8<DT> raw[kTileRows];
  auto fetch = [&](int64_t s0) {
    const char* at = x + s0 * P.l * P.ld_x;
    const int64_t left = all_rows - s0 * P.l;
    const int here = left < tile_rows ? static_cast<int>(left < 0 ? 0 : left) : tile_rows;
#pragma unroll
    for (int u = 0; u < kTileRows; ++u) {
      const int row = ry + u * P.rows;
      raw[u] = Vec8<DT>{};
      if (on && row < here) load_pack(raw[u], at + row * P.ld_x);
    }
  };
  const int64_t s_first = static_cast<int64_t>(part) * P.samples;
  fetch(s_first);
  for (int64_t s0 = s_first; s0 < P.n; s0 += step) {
    const int64_t row0 = s0 * P.l;
    const int64_t left = all_rows - row0;
    const int here = left < tile_rows ? static_cast<int>(left) : tile_rows;
    F2 v[kTileRows][4];
#pragma unroll
    for (int u = 0; u < kTileRows; ++u) unpack_pairs(raw[u], v[u]);
    fetch(s0 + step);
    float mean[kTileRows], rstd[kTileRows];
#pragma unroll
    for (int u = 0; u < kTileRows; ++u) mean[u] = 0.f;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      // pass 0: the mean (LayerNorm); pass 1: the mean square around it
      if (pass == 0 && !ln) continue;
#pragma unroll
      for (int u = 0; u < kTileRows; ++u)
        if (ry < P.rows)
          dyn[(ry + u * P.rows) * P.cols + cx] =
              pass == 0 ? pair_sum(v[u]) : spread_sum(v[u], mean[u]);
      __syncthreads();
      const int lane = threadIdx.x % P.lanes, teams = blockDim.x / P.lanes;
      for (int p0 = 0; p0 < pairs; p0 += teams) {
        const int p = p0 + threadIdx.x / P.lanes;
        float w = 0.f;
        if (p < pairs) {
          const int s = p / slab_groups;
          const float* at = dyn + s * l * P.cols + (p - s * slab_groups) * P.q;
          for (int i = 0; i < l; ++i, at += P.cols)
            for (int j = lane; j < P.q; j += P.lanes) w += at[j];
        }
        w = lanes_sum(w, P.lanes);
        if (p < pairs && lane == 0)
          stat[pass * pairs + p] = pass == 0 ? mean_of(w, P.count, P.count_inv)
                                             : rsqrtf(w * P.count_inv + P.eps);
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kTileRows; ++u) (pass == 0 ? mean : rstd)[u] = stat[pass * pairs + pair[u]];
    }
    char* to = out + row0 * P.ld_out;
#pragma unroll
    for (int u = 0; u < kTileRows; ++u) {
      const int row = ry + u * P.rows;
      if (!on || row >= here) continue;
      store_pack(to + row * P.ld_out, norm_act<DT>(v[u], rstd[u], col, silu));
      if (leads[u]) {
        const int64_t at = (s0 + row / l) * P.groups + group;
        if (ln) P.mean[r][at] = mean[u];
        P.rstd[r][at] = rstd[u];
      }
    }
    __syncthreads();                           // the next tile's sums replace this one's statistics
  }
}

// A cluster's statistics of its sample's slab from `sums`, (mean, M2) of each
// thread's values: stat[g] = (mean, rstd).  `blocks`: the sample's rows dealt to
// the blocks, `lanes`: this block's to its threads' rows.
__device__ __forceinline__ void join_moments(const GroupNormParams& P, int C, int rank, int slab,
                                             int r, int64_t sample, const Deal& blocks,
                                             const Deal& lanes, const float2* sums,
                                             float2* joined, float2* stat) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int slab_groups = P.cols / P.q;
  const bool ln = P.norm == SP_NORM_LAYERNORM;
  const float block_count = static_cast<float>(blocks.count(rank)) * 8.f * P.q;
  auto put = [&](int g, float m, float v) {
    const float2 st = make_float2(m, rsqrtf(v * P.count_inv + P.eps));
    stat[g] = st;
    const int group = slab * slab_groups + g;
    if (rank == 0 && group < P.groups) {
      if (ln) P.mean[r][sample * P.groups + group] = st.x;
      P.rstd[r][sample * P.groups + group] = st.y;
    }
  };
  __syncthreads();
  if (C > 1) cluster_wait();                   // the partners run: their shared memory is there
  // one warp a group
  for (int g = warp; g < slab_groups; g += nw) {
    float s = 0.f, v = 0.f;
    if (ln) group_entries(P, g, [&](int y, int at) { s += 8.f * lanes.count(y) * sums[at].x; });
    const float m = ln && block_count > 0.f ? warp_sum(s) / block_count : 0.f;
    group_entries(P, g, [&](int y, int at) {
      const float d = sums[at].x - m;
      v += sums[at].y + 8.f * lanes.count(y) * d * d;
    });
    v = warp_sum(v);
    if (C == 1) {
      if (lane == 0) put(g, m, v);
    } else if (lane < C) {
      const uint32_t to = cluster_map(&joined[rank * slab_groups + g], lane);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(m), "f"(v)
                   : "memory");
    }
  }
  if (C > 1) {
    cluster_sync_all();
    for (int g = threadIdx.x; g < slab_groups; g += blockDim.x) {
      float m = 0.f, v = 0.f;
      for (int k = 0; k < C; ++k)
        m += joined[k * slab_groups + g].x * static_cast<float>(blocks.count(k));
      m /= static_cast<float>(P.l);
      for (int k = 0; k < C; ++k) {
        const float2 w = joined[k * slab_groups + g];
        const float d = w.x - m;
        v += w.y + static_cast<float>(blocks.count(k)) * 8.f * P.q * d * d;
      }
      put(g, m, v);
    }
  }
  __syncthreads();
}

// Held: a block keeps its sample's slab in registers, and takes one sample after
// the other.
template <int DT>
__global__ void __launch_bounds__(256, kHeldBlocks) group_held_fwd_kernel(const GroupNormParams P) {
  constexpr int E = ElemSize<DT>::value, kMost = kHold<DT>;
  extern __shared__ float2 sums[];             // [threads] mean, M2
  pdl_wait();
  const int cx = threadIdx.x % P.cols, ry = threadIdx.x / P.cols;
  const int slab = blockIdx.x % P.slabs;
  const int r = blockIdx.x / P.slabs % P.t;
  const int part = static_cast<int>(blockIdx.x) / (P.slabs * P.t);
  const int vec = slab * P.cols + cx;
  const bool on = ry < P.rows && vec * 8 < P.c;
  const bool ln = P.norm == SP_NORM_LAYERNORM, silu = P.act == SP_ACT_SILU;
  float2* stat = sums + blockDim.x;            // [slab groups] mean, rstd
  const Deal blocks(static_cast<int>(P.l), 1), lanes(static_cast<int>(P.l), P.rows);
  const int mine = on ? lanes.count(ry) : 0;
  const int64_t row0 = part * P.l + ry;
  const char* x = P.x[r] + row0 * P.ld_x + static_cast<int64_t>(vec) * 8 * E;
  char* out = P.out[r] + row0 * P.ld_out + static_cast<int64_t>(vec) * 8 * E;
  const int64_t step_x = P.ld_x * P.rows, step_out = P.ld_out * P.rows;
  const int64_t skip_x = P.parts * P.l * P.ld_x, skip_out = P.parts * P.l * P.ld_out;
  Column<DT> col;
  col.read(P, static_cast<int64_t>(r) * P.c + vec * 8, on);
  const float count = 8.f * static_cast<float>(mine), each = mine > 0 ? 1.f / count : 0.f;
  for (int64_t sample = part; sample < P.n; sample += P.parts, x += skip_x, out += skip_out) {
    Vec8<DT> raw[kMost];
    const char* from = x;
#pragma unroll
    for (int u = 0; u < kMost; ++u, from += step_x)
      if (u < mine) load_pack(raw[u], from);
    float2 mom = make_float2(0.f, 0.f);
    if (ln) {
#pragma unroll
      for (int u = 0; u < kMost; ++u)
        if (u < mine) {
          F2 v[4];
          unpack_pairs(raw[u], v);
          mom.x += pair_sum(v);
        }
      mom.x = mean_of(mom.x, count, each);
    }
#pragma unroll
    for (int u = 0; u < kMost; ++u)
      if (u < mine) {
        F2 v[4];
        unpack_pairs(raw[u], v);
        mom.y += spread_sum(v, mom.x);
      }
    if (ry < P.rows) sums[threadIdx.x] = mom;
    join_moments(P, 1, 0, slab, r, sample, blocks, lanes, sums, nullptr, stat);
    const float2 st = stat[on ? cx / P.q : 0];
    char* to = out;
#pragma unroll
    for (int u = 0; u < kMost; ++u, to += step_out)
      if (u < mine) {
        F2 v[4];
        unpack_pairs(raw[u], v);
        centre(v, st.x);
        store_pack(to, norm_act<DT>(v, st.y, col, silu));
      }
  }
}

// One cluster per (sample, rank, slab).  WIDE: blocks of up to 512 threads, or few
// enough that an SM need not hold three: more registers, more vectors on their way
// (10 clusters of 16, 32,771 rows: 52 us against 56).
template <int DT, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kGroupThreads : 256, WIDE ? 1 : kUnitBlocks)
group_unit_fwd_kernel(const GroupNormParams P) {
  constexpr int E = ElemSize<DT>::value, kRing = WIDE ? kWideRing<DT> : kUnitRing<DT>;
  extern __shared__ float2 sums[];             // [threads] mean, M2
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
  float2* joined = sums + blockDim.x;          // [cluster][slab groups] mean, M2 of each block
  float2* stat = joined + C * (P.cols / P.q);  // [slab groups] mean, rstd
  // this block's rows of the sample, and this thread's: ry, ry + rows, ...
  const Deal blocks(static_cast<int>(P.l), C);
  const int b0 = blocks.first(rank), block_rows = blocks.count(rank);
  const Deal lanes(block_rows, P.rows);
  const int mine = on ? lanes.count(ry) : 0;
  const int64_t row0 = sample * P.l + b0 + ry;
  const char* x = P.x[r] + row0 * P.ld_x + static_cast<int64_t>(vec) * 8 * E;
  const int64_t step_x = P.ld_x * P.rows, step_out = P.ld_out * P.rows;
  Moments mom;
  // a vector's place is filled again as soon as it is used
  Vec8<DT> raw[kRing];
  const char* from = x;
  auto fetch = [&](int u, int i, bool again) {
    if (i < mine) {
      if (again) load_again<DT>(raw[u], from);
      else load_pack(raw[u], from);
    }
    from += step_x;
  };
#pragma unroll
  for (int u = 0; u < kRing; ++u) fetch(u, u, true);
  for (int i0 = 0; i0 < mine; i0 += kRing) {
#pragma unroll
    for (int u = 0; u < kRing; ++u) {
      F2 v[4];
      unpack_pairs(raw[u], v);
      if (i0 + u < mine) mom.add(v, ln);
      fetch(u, i0 + kRing + u, true);
    }
    if (mom.n >= kStretch - kRing) mom.join(ln);
  }
  mom.join(ln);
  from = x;
#pragma unroll
  for (int u = 0; u < kRing; ++u) fetch(u, u, false);
  if (ry < P.rows) sums[threadIdx.x] = make_float2(mom.mean, mom.m2);
  join_moments(P, C, rank, slab, r, sample, blocks, lanes, sums, joined, stat);
  if (!on) return;
  const float2 st = stat[cx / P.q];
  Column<DT> col;
  col.read(P, static_cast<int64_t>(r) * P.c + vec * 8, on);
  fold_rstd(col, st.y);
  char* out = P.out[r] + row0 * P.ld_out + static_cast<int64_t>(vec) * 8 * E;
  for (int i0 = 0; i0 < mine; i0 += kRing) {
#pragma unroll
    for (int u = 0; u < kRing; ++u, out += step_out) {
      F2 v[4];
      unpack_pairs(raw[u], v);
      fetch(u, i0 + kRing + u, false);
      centre(v, st.x);
      if (i0 + u < mine) store_pack(out, norm_act<DT, true>(v, st.y, col, silu));
    }
  }
}

static int div_up(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

GroupShape group_norm_shape(int64_t n, int64_t l, int c, int groups, int t, int dtype, bool bwd) {
  GroupShape s{};
  const int size = dtype == SP_F32 ? 4 : 2;
  const int nvec = c / 8, q = nvec / groups;
  const int sms = device_sm_count();
  const int held_rows = bwd ? kBackTileRows : kTileRows;
  auto fit_cols = [&](int most) {
    int g = most / q;
    if (g < 1) g = 1;
    if (g > groups) g = groups;
    s.cols = g * q;
    s.slabs = div_up(groups, g);
  };
  s.cluster = 1;
  if (l == 1) {
    // rows: whole groups of up to 32 vectors a warp, wider ones a team of warps
    s.form = kRowForm;
    s.mode = q > 32 ? kSumTeam : (q & (q - 1)) == 0 ? kSumLanes : kSumWarp;
    fit_cols(32);
    const int team = (s.cols + 31) / 32;
    s.rows = team < kRowWarps ? kRowWarps / team : 1;
    s.threads = s.rows * team * 32;
    const int row_rows = bwd ? kBackRowRows : size == 4 ? kRowRows<SP_F32> : kRowRows<SP_BF16>;
    const int blocks = bwd ? kBackRowBlocks : size == 4 ? kRowBlocks<SP_F32> : kRowBlocks<SP_BF16>;
    const int64_t tiles = div_up(n, static_cast<int64_t>(s.rows) * row_rows);
    const int64_t cap = static_cast<int64_t>(sms) * blocks / (s.slabs * t);
    s.parts = cap < 1 ? 1 : tiles < cap ? tiles : cap;
    s.smem = bwd ? static_cast<size_t>(s.rows) * s.cols * 17 * 4 : 0;
    return s;
  }
  static const int kClusters[] = {1, 2, 3, 4, 6, 8, 10, 12, kGroupMaxCluster};
  auto narrow = [&]() {
    // narrow slabs of at least 128 bytes of a row, whole 32-byte sectors where
    // that takes two groups at most, and many rows abreast
    fit_cols(q >= 8 ? q : (8 + q - 1) / q * q);
    if (s.cols % 2 != 0 && 2 * s.cols <= (nvec < kGroupThreads ? nvec : kGroupThreads))
      fit_cols(2 * s.cols);
    s.rows = 256 / s.cols > 0 ? 256 / s.cols : 1;
  };
  // held: samples of some rows whose slab, 160 to 1024 vectors, fits the registers
  // of a block of up to 256 threads, as few threads as hold it (blocks of one warp
  // overlap best) unless that leaves the SMs half empty.  Fewer vectors a sample
  // than that hide the joins' latency badly, more leave the loads without
  // overlap.  (64 MB of bf16 in 8 groups of 512 channels, held against the other
  // forms, forward and backward in us: samples of 12 rows 86, 87 against 70, 88;
  // 16 rows 69, 77 against 65, 78; 24 rows 53, 72 against 97, 317; 48 rows 40, 75
  // against 133, 178; 128 rows 66, 86 against 64, 96; 200 rows 56, 110 against
  // 55, 81.)
  const int hold = bwd ? (size == 4 ? kBackHold<SP_F32> : kBackHold<SP_BF16>)
                       : (size == 4 ? kHold<SP_F32> : kHold<SP_BF16>);
  narrow();
  if (l * s.cols >= 160 && l * s.cols <= 1024 && s.cols <= 256 &&
      l <= static_cast<int64_t>(s.rows) * hold) {
    s.form = kHeldForm;
    const int64_t units = n * t * s.slabs;
    const int most = s.rows;
    s.rows = div_up(l, hold);
    if (s.rows < 32 / s.cols) s.rows = 32 / s.cols;
    while (2 * s.rows <= most && units * s.rows * s.cols < int64_t(256) * sms) s.rows *= 2;
    s.threads = (s.rows * s.cols + 31) / 32 * 32;
    const int64_t cap = static_cast<int64_t>(sms) * kHeldBlocks * (256 / s.threads) / (s.slabs * t);
    s.parts = cap < 1 ? 1 : n < cap ? n : cap;
    s.smem = (static_cast<size_t>(s.threads) + s.cols / q) * 8;
    if (bwd) {
      const size_t part = static_cast<size_t>(s.rows) * s.cols * 17 * 4;
      if (s.smem < part) s.smem = part;
    }
    return s;
  }
  // tiles while a block of up to 256 threads holds a whole sample in its registers
  // (16,384 samples of 4 rows of 8 groups of 64 channels: 51 us, held by blocks of
  // their own 220)
  fit_cols(256);
  s.rows = 256 / s.cols > 0 ? 256 / s.cols : 1;
  if (l > static_cast<int64_t>(s.rows) * held_rows && l * q < 160 && q <= 32) {
    fit_cols(32);     // fewer columns abreast: more rows of a sample in one block
    s.rows = 256 / s.cols;
  }
  if (l <= static_cast<int64_t>(s.rows) * held_rows) {
    s.form = kTileForm;
    s.threads = (s.rows * s.cols + 31) / 32 * 32;
    s.samples = static_cast<int>(s.rows * held_rows / l);
    // fewer samples a tile while that leaves SMs without one
    while (s.samples > 1 && static_cast<int64_t>(s.slabs) * t * div_up(n, s.samples) < 2 * sms)
      s.samples = (s.samples + 1) / 2;
    const int64_t tiles = (n + s.samples - 1) / s.samples;
    const int64_t cap = static_cast<int64_t>(sms) * 2 / (s.slabs * t);
    s.parts = cap < 1 ? 1 : tiles < cap ? tiles : cap;
    const int pairs = s.samples * (s.cols / q);
    s.lanes = 1;
    while (s.lanes < 32 && s.lanes < q && pairs * s.lanes < s.threads) s.lanes *= 2;
    const int sums = bwd ? 2 : 1;
    s.smem = (static_cast<size_t>(s.rows) * held_rows * s.cols * sums + 2 * pairs) * 4;
    if (bwd) {
      const size_t part = static_cast<size_t>(s.rows) * s.cols * 17 * 4;
      if (s.smem < part) s.smem = part;
    }
    return s;
  }
  s.form = kUnitForm;
  narrow();
  const int64_t units = n * t * s.slabs;
  // Few long slabs, whose longest clusters leave SMs free, take blocks of twice the
  // threads.  (Forward and backward in us: 65,536 rows of one group of 64 29, 48
  // against 41, 62; 20,000 float32 rows of one of 320 86, 122 against 99, 160.  From 10
  // units on the longest clusters of such blocks do not all fit: 32,771 rows of 2 x
  // 640 in 5 groups 76, 81 against 56, 78.)
  if (units * kGroupMaxCluster * 10 <= int64_t(9) * sms && 2 * s.cols <= kGroupThreads &&
      l >= int64_t(64) * s.rows)
    s.rows = kGroupThreads / s.cols;
  s.threads = (s.rows * s.cols + 31) / 32 * 32;
  // Of the clusters that leave what the blocks at work read inside L2 (129 MB) the
  // one with the least waves x (3 us + 0.2 us a vector of a thread): short rows of
  // waves that are full.  (Forward and backward in us, bf16.  32 samples of 1024 x
  // 320 in 5 groups: C = 1 17, 28; 2 14, 29; 3 18, 27; 6 21, 37.  8 of 4096 x 1280 in
  // 32: 1 68, 111; 2 49, 78; 3 45, 95; 4 52, 79; 6 45, 81; 12 53, 93.  8 ranks' 4 of
  // 2048 x 2048 in 8: 1 146, 228; 3 134, 233; 6 130, 230; 16 195, 311.)
  const int64_t resident =
      static_cast<int64_t>(s.threads > 256 ? 1 : bwd ? kBackUnitBlocks : kUnitBlocks) * sms;
  const int64_t slab_bytes = l * s.cols * 8 * size * (bwd ? 2 : 1);
  double best = 0;
  for (int cl : kClusters) {
    if (cl > 1 && l < static_cast<int64_t>(cl) * s.rows) break;
    // long clusters leave some SMs without a block: they lie within one part of the GPU
    int64_t fit = resident * (cl < 6 ? 95 : cl < kGroupMaxCluster ? 85 : 70) / (100 * cl);
    if (fit < 1) fit = 1;
    const int64_t at_once = fit < units ? fit : units;
    const bool inside = at_once * slab_bytes <= int64_t(128) << 20;
    const double time = static_cast<double>((units + fit - 1) / fit) *
                        (3.0 + 0.2 * static_cast<double>(l) / (cl * s.rows));
    if (best > 0 && (!inside || time >= best)) continue;
    best = inside ? time : 0;                  // a later one replaces what L2 does not hold
    s.cluster = cl;
  }
  s.smem = (static_cast<size_t>(s.threads) + static_cast<size_t>(s.cluster + 1) * (s.cols / q)) * 8;
  if (bwd) {
    const size_t part = static_cast<size_t>(s.rows) * s.cols * 17 * 4;
    if (s.smem < part) s.smem = part;
  }
  s.parts = n * s.cluster;
  s.roomy = units * s.cluster * 10 <= int64_t(14) * sms;
  return s;
}

static void fill_shape(GroupNormParams* p, const GroupShape& s) {
  p->q = p->c / 8 / p->groups;
  p->cols = s.cols;
  p->slabs = s.slabs;
  p->rows = s.rows;
  p->samples = s.samples;
  p->lanes = s.lanes;
  p->parts = s.parts;
  p->cluster = s.cluster;
}

cudaError_t launch_group(const void* fn, GroupNormParams* p, const GroupShape& s, cudaStream_t st) {
  fill_shape(p, s);
  void* args[] = {p};
  int fit = 1;
  const cudaError_t e = s.form == kUnitForm ? max_clusters(fn, s.threads, s.smem, s.cluster, &fit)
                             : ensure_smem_attr(fn, s.smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = static_cast<int64_t>(s.slabs) * p->t * s.parts;
  if (fit < 1 || blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(fn, dim3(static_cast<unsigned>(blocks)), dim3(s.threads), s.smem, args, st,
                    s.cluster);
}

template <int DT>
static const void* fwd_fn(const GroupShape& s) {
  if (s.form == kRowForm)
    return s.mode == kSumLanes  ? reinterpret_cast<const void*>(&group_row_fwd_kernel<DT, kSumLanes>)
           : s.mode == kSumWarp ? reinterpret_cast<const void*>(&group_row_fwd_kernel<DT, kSumWarp>)
                                : reinterpret_cast<const void*>(&group_row_fwd_kernel<DT, kSumTeam>);
  if (s.form == kTileForm) return reinterpret_cast<const void*>(&group_tile_fwd_kernel<DT>);
  if (s.form == kHeldForm) return reinterpret_cast<const void*>(&group_held_fwd_kernel<DT>);
  return s.threads > 256 || s.roomy ? reinterpret_cast<const void*>(&group_unit_fwd_kernel<DT, true>)
                         : reinterpret_cast<const void*>(&group_unit_fwd_kernel<DT, false>);
}

cudaError_t launch_group_norm_fwd(GroupNormParams p, int dtype, cudaStream_t st) {
  const GroupShape s = group_norm_shape(p.n, p.l, p.c, p.groups, p.t, dtype, false);
  const void* fn = dtype == SP_BF16  ? fwd_fn<SP_BF16>(s)
                   : dtype == SP_F16 ? fwd_fn<SP_F16>(s)
                                     : fwd_fn<SP_F32>(s);
  return launch_group(fn, &p, s, st);
}

}  // namespace spb
