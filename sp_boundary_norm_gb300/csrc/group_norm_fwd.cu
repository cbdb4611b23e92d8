// Group norm with an activation, forward (the forms are described in
// group_norm.cuh), and the split of a call over the GPU for both directions.
#include "group_norm.cuh"

namespace spb {

constexpr int kTileRows = 4;    // vectors a thread holds (tiles)
constexpr int kUnitBatch = 8;   // vectors a thread reads at once (units)

// SHFL: one row a sample and a power of two up to 32 vectors a group: the sums
// stay within neighbouring lanes.  Else through shared memory.
template <int DT, bool SHFL>
__global__ void __launch_bounds__(kGroupThreads) group_tile_fwd_kernel(const GroupNormParams P) {
  constexpr int E = ElemSize<DT>::value;
  extern __shared__ float dyn[];               // [tile rows][cols] sums, then [pairs] statistics
  pdl_wait();
  const int cx = threadIdx.x % P.cols, ry = threadIdx.x / P.cols;
  const int slab = blockIdx.x % P.slabs;
  const int r = blockIdx.x / P.slabs % P.t;
  const int64_t part = blockIdx.x / (P.slabs * P.t);
  const int vec = slab * P.cols + cx;
  const bool on = ry < P.rows && vec * 8 < P.c;
  const bool ln = P.norm == SP_NORM_LAYERNORM, silu = P.act == SP_ACT_SILU;
  Column<DT> col;
  col.read(P, static_cast<int64_t>(r) * P.c + vec * 8, on);
  const char* x = P.x[r] + static_cast<int64_t>(vec) * 8 * E;
  char* out = P.out[r] + static_cast<int64_t>(vec) * 8 * E;
  const int tile_rows = static_cast<int>(P.samples * P.l);
  const int slab_groups = P.cols / P.q;
  const int pairs = P.samples * slab_groups;
  float* stat = dyn + P.rows * kTileRows * P.cols;     // mean then rstd of each pair
  const int group = vec / P.q;

  for (int64_t s0 = part * P.samples; s0 < P.n; s0 += P.parts * P.samples) {
    const int64_t row0 = s0 * P.l;
    const int64_t left = P.n * P.l - row0;
    const int here = left < tile_rows ? static_cast<int>(left) : tile_rows;
    Vec8<DT> raw[kTileRows];
    float mean[kTileRows], rstd[kTileRows];
#pragma unroll
    for (int u = 0; u < kTileRows; ++u) {
      raw[u] = Vec8<DT>{};
      const int row = ry + u * P.rows;
      if (on && row < here) load_pack(raw[u], x + (row0 + row) * P.ld_x);
    }
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      // pass 0: the mean (LayerNorm); pass 1: the mean square around it
      if (pass == 0 && !ln) {
#pragma unroll
        for (int u = 0; u < kTileRows; ++u) mean[u] = 0.f;
        continue;
      }
      float sum[kTileRows];
#pragma unroll
      for (int u = 0; u < kTileRows; ++u) {
        float f[8];
        unpack(raw[u], f);
        sum[u] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = pass == 0 ? f[i] : f[i] - mean[u];
          sum[u] = pass == 0 ? sum[u] + d : fmaf(d, d, sum[u]);
        }
        if constexpr (SHFL) sum[u] = lanes_sum(sum[u], P.q);
      }
      if constexpr (!SHFL) {
#pragma unroll
        for (int u = 0; u < kTileRows; ++u)
          if (ry < P.rows) dyn[(ry + u * P.rows) * P.cols + cx] = sum[u];
        __syncthreads();
        const int lane = threadIdx.x % P.lanes, step = blockDim.x / P.lanes;
        for (int p0 = 0; p0 < pairs; p0 += step) {
          const int p = p0 + threadIdx.x / P.lanes;
          float v = 0.f;
          if (p < pairs) {
            const int s = p / slab_groups, g = p - s * slab_groups;
            const int terms = static_cast<int>(P.l) * P.q;
            for (int e = lane; e < terms; e += P.lanes) {
              const int i = e / P.q;
              v += dyn[(s * static_cast<int>(P.l) + i) * P.cols + g * P.q + (e - i * P.q)];
            }
          }
          v = lanes_sum(v, P.lanes) * P.count_inv;
          if (p < pairs && lane == 0) stat[pass * pairs + p] = pass == 0 ? v : rsqrtf(v + P.eps);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kTileRows; ++u) {
          const int row = ry + u * P.rows;
          const int p = row < tile_rows
                            ? row / static_cast<int>(P.l) * slab_groups + cx / P.q : 0;
          (pass == 0 ? mean : rstd)[u] = stat[pass * pairs + p];
        }
      } else {
#pragma unroll
        for (int u = 0; u < kTileRows; ++u) {
          if (pass == 0) mean[u] = sum[u] * P.count_inv;
          else rstd[u] = rsqrtf(sum[u] * P.count_inv + P.eps);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kTileRows; ++u) {
      const int row = ry + u * P.rows;
      if (!on || row >= here) continue;
      float f[8];
      unpack(raw[u], f);
      Vec8<DT> o;
      norm_act<DT>(f, mean[u], rstd[u], col, silu, o);
      store_pack(out + (row0 + row) * P.ld_out, o);
      if (vec % P.q == 0 && row % P.l == 0) {
        const int64_t at = (s0 + row / static_cast<int>(P.l)) * P.groups + group;
        if (ln) P.mean[r][at] = mean[u];
        P.rstd[r][at] = rstd[u];
      }
    }
    if constexpr (!SHFL) __syncthreads();   // the next tile's sums replace this one's statistics
  }
}

// One cluster per (sample, rank, slab).
template <int DT>
__global__ void __launch_bounds__(kGroupThreads) group_unit_fwd_kernel(const GroupNormParams P) {
  constexpr int E = ElemSize<DT>::value;
  extern __shared__ uint4 kept[];              // [keep][threads] vectors, then the sums below
  const int C = P.cluster, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  if (C > 1) cluster_sync_all();               // the partners run: their shared memory is there
  pdl_wait();
  const int cx = threadIdx.x % P.cols, ry = threadIdx.x / P.cols;
  int unit = static_cast<int>(blockIdx.x) / C;
  const int slab = unit % P.slabs;
  unit /= P.slabs;
  const int r = unit % P.t;
  const int64_t sample = unit / P.t;
  const int vec = slab * P.cols + cx;
  const bool on = ry < P.rows && vec * 8 < P.c;
  const bool ln = P.norm == SP_NORM_LAYERNORM, silu = P.act == SP_ACT_SILU;
  const int slab_groups = P.cols / P.q;
  constexpr int kPer = E == 4 ? 2 : 1;         // 16-byte pieces of a vector
  float2* sums = reinterpret_cast<float2*>(kept + static_cast<int64_t>(P.keep) * kPer * blockDim.x);
  float2* joined = sums + blockDim.x;          // [cluster][slab groups] mean, M2 of each block
  float2* stat = joined + C * slab_groups;     // [slab groups] mean, rstd
  Column<DT> col;
  col.read(P, static_cast<int64_t>(r) * P.c + vec * 8, on);
  // this block's rows of the sample, and this thread's: ry, ry + rows, ...
  const int64_t b0 = P.l * rank / C, b1 = P.l * (rank + 1) / C;
  const int mine = b1 - b0 > ry ? static_cast<int>((b1 - b0 - ry + P.rows - 1) / P.rows) : 0;
  const int64_t row0 = sample * P.l + b0 + ry;
  const char* x = P.x[r] + row0 * P.ld_x + static_cast<int64_t>(vec) * 8 * E;
  char* out = P.out[r] + row0 * P.ld_out + static_cast<int64_t>(vec) * 8 * E;
  const int64_t step_x = P.ld_x * P.rows, step_out = P.ld_out * P.rows;

  // (count, mean, M2) of the thread's values, batch by batch
  float cnt = 0.f, mean = 0.f, m2 = 0.f;
  for (int i0 = 0; on && i0 < mine; i0 += kUnitBatch) {
    Vec8<DT> raw[kUnitBatch];
#pragma unroll
    for (int u = 0; u < kUnitBatch; ++u) {
      raw[u] = Vec8<DT>{};
      if (i0 + u < mine) load_pack(raw[u], x + (i0 + u) * step_x);
    }
    const int nb = (mine - i0 < kUnitBatch ? mine - i0 : kUnitBatch);
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < kUnitBatch; ++u) {
      float f[8];
      unpack(raw[u], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) s += f[i];
      if (i0 + u < P.keep && u < nb) {
        uint4* to = kept + static_cast<int64_t>(i0 + u) * kPer * blockDim.x + threadIdx.x;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          to[k * blockDim.x] = make_uint4(raw[u].w[4 * k], raw[u].w[4 * k + 1],
                                          raw[u].w[4 * k + 2], raw[u].w[4 * k + 3]);
      }
    }
    const float nf = 8.f * static_cast<float>(nb);
    const float mb = ln ? __fdividef(s, nf) : 0.f;
    float q2 = 0.f;
#pragma unroll
    for (int u = 0; u < kUnitBatch; ++u) {
      if (u < nb) {
        float f[8];
        unpack(raw[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = f[i] - mb;
          q2 = fmaf(d, d, q2);
        }
      }
    }
    const float d = mb - mean, all = cnt + nf;
    mean += d * __fdividef(nf, all);
    m2 += q2 + d * d * __fdividef(cnt * nf, all);
    cnt = all;
  }
  // the block's mean and M2 of each group of the slab, one warp a group
  if (ry < P.rows) sums[threadIdx.x] = make_float2(mean, m2);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int terms = P.rows * P.q;
  auto rows_of = [&](int y) {
    return b1 - b0 > y ? static_cast<float>((b1 - b0 - y + P.rows - 1) / P.rows) * 8.f : 0.f;
  };
  const float block_count = static_cast<float>(b1 - b0) * 8.f * P.q;
  for (int g = warp; g < slab_groups; g += nw) {
    float s = 0.f;
    if (ln)
      for (int e = lane; e < terms; e += 32) {
        const int y = e / P.q;
        s += rows_of(y) * sums[y * P.cols + g * P.q + (e - y * P.q)].x;
      }
    const float m = block_count > 0.f ? warp_sum(s) / block_count : 0.f;
    float v = 0.f;
    for (int e = lane; e < terms; e += 32) {
      const int y = e / P.q;
      const float2 w = sums[y * P.cols + g * P.q + (e - y * P.q)];
      const float d = w.x - m;
      v += w.y + rows_of(y) * d * d;
    }
    v = warp_sum(v);
    if (C == 1) {
      if (lane == 0) joined[g] = make_float2(m, v);
    } else if (lane < C) {
      const uint32_t to = cluster_map(&joined[rank * slab_groups + g], lane);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(m), "f"(v)
                   : "memory");
    }
  }
  if (C > 1) cluster_sync_all(); else __syncthreads();
  for (int g = threadIdx.x; g < slab_groups; g += blockDim.x) {
    float m = 0.f, v = 0.f;
    for (int k = 0; k < C; ++k)
      m += joined[k * slab_groups + g].x *
           static_cast<float>(P.l * (k + 1) / C - P.l * k / C);
    m /= static_cast<float>(P.l);
    for (int k = 0; k < C; ++k) {
      const float2 w = joined[k * slab_groups + g];
      const float d = w.x - m;
      v += w.y + static_cast<float>(P.l * (k + 1) / C - P.l * k / C) * 8.f * P.q * d * d;
    }
    const float2 st = make_float2(m, rsqrtf(v * P.count_inv + P.eps));
    stat[g] = st;
    const int group = slab * slab_groups + g;
    if (rank == 0 && group < P.groups) {
      if (ln) P.mean[r][sample * P.groups + group] = st.x;
      P.rstd[r][sample * P.groups + group] = st.y;
    }
  }
  __syncthreads();
  if (!on) return;
  const float2 st = stat[cx / P.q];
  for (int i0 = 0; i0 < mine; i0 += kUnitBatch) {
    Vec8<DT> raw[kUnitBatch];
#pragma unroll
    for (int u = 0; u < kUnitBatch; ++u) {
      const int i = i0 + u;
      if (i >= mine) continue;
      if (i < P.keep) {
        const uint4* from = kept + static_cast<int64_t>(i) * kPer * blockDim.x + threadIdx.x;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const uint4 v = from[k * blockDim.x];
          raw[u].w[4 * k] = v.x;
          raw[u].w[4 * k + 1] = v.y;
          raw[u].w[4 * k + 2] = v.z;
          raw[u].w[4 * k + 3] = v.w;
        }
      } else {
        load_pack(raw[u], x + i * step_x);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnitBatch; ++u) {
      if (i0 + u >= mine) continue;
      float f[8];
      unpack(raw[u], f);
      Vec8<DT> o;
      norm_act<DT>(f, st.x, st.y, col, silu, o);
      store_pack(out + (i0 + u) * step_out, o);
    }
  }
}

static int div_up(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

GroupShape group_norm_shape(int64_t n, int64_t l, int c, int groups, int t, int dtype, bool bwd) {
  GroupShape s{};
  const int size = dtype == SP_F32 ? 4 : 2;
  const int nvec = c / 8, q = nvec / groups;
  const int sms = device_sm_count();
  // tiles while a block of up to 256 threads holds a whole sample in its registers
  auto fit_cols = [&](int most) {
    int g = most / q;
    if (g < 1) g = 1;
    if (g > groups) g = groups;
    s.cols = g * q;
    s.slabs = div_up(groups, g);
  };
  fit_cols(256);
  s.rows = 256 / s.cols > 0 ? 256 / s.cols : 1;
  if (l > static_cast<int64_t>(s.rows) * kTileRows && l <= 64 && q <= 32) {
    fit_cols(32);     // fewer columns abreast: more rows of a sample in one block
    s.rows = 256 / s.cols;
  }
  s.tile = l <= static_cast<int64_t>(s.rows) * kTileRows;
  s.cluster = 1;
  if (s.tile) {
    s.threads = (s.rows * s.cols + 31) / 32 * 32;
    s.shuffle = l == 1 && q <= 32 && (q & (q - 1)) == 0;
    s.samples = static_cast<int>(s.rows * kTileRows / l);
    // fewer samples a tile while that leaves SMs without one
    while (s.samples > 1 && s.rows > 1 &&
           static_cast<int64_t>(s.slabs) * t * div_up(n, s.samples) < 2 * sms) {
      s.samples = (s.samples + 1) / 2;
    }
    const int64_t tiles = (n + s.samples - 1) / s.samples;
    const int64_t cap = (static_cast<int64_t>(sms) * 8 + s.slabs * t - 1) / (s.slabs * t);
    s.parts = tiles < cap ? tiles : cap;
    const int pairs = s.samples * (s.cols / q);
    s.lanes = 1;
    while (s.lanes < 32 && s.lanes < l * q && pairs * s.lanes < s.threads) s.lanes *= 2;
    const int sums = bwd ? 2 : 1;
    s.smem = s.shuffle ? 0
                       : (static_cast<size_t>(s.rows) * kTileRows * s.cols * sums + 2 * pairs) * 4;
    if (bwd) {
      const size_t part = static_cast<size_t>(s.rows) * s.cols * 17 * 4;
      if (s.smem < part) s.smem = part;
    }
    return s;
  }
  // units: narrow slabs (at least 128 bytes of a row), many rows abreast
  fit_cols(q >= 8 ? q : 16);
  s.rows = 256 / s.cols > 0 ? 256 / s.cols : 1;
  s.threads = (s.rows * s.cols + 31) / 32 * 32;
  const int64_t units = n * t * s.slabs;
  while (s.cluster < kGroupMaxCluster && units * s.cluster < 4 * sms &&
         static_cast<int64_t>(s.rows) * kUnitBatch * s.cluster < l)
    s.cluster *= 2;
  const int64_t need = (l + static_cast<int64_t>(s.rows) * s.cluster - 1) /
                       (static_cast<int64_t>(s.rows) * s.cluster);
  const int slab_groups = s.cols / q;
  const size_t fixed = static_cast<size_t>(s.threads) * 8 +
                       static_cast<size_t>(s.cluster + 1) * slab_groups * 8;
  const size_t vec = static_cast<size_t>(s.threads) * 8 * size * (bwd ? 2 : 1);
  size_t room = 100 * 1024;
  if (room < fixed) room = fixed;
  int64_t keep = static_cast<int64_t>((room - fixed) / vec);
  if (keep > need) keep = need;
  s.keep = static_cast<int>(keep);
  s.smem = s.keep * vec + fixed;
  if (bwd) {
    const size_t part = static_cast<size_t>(s.rows) * s.cols * 17 * 4;
    if (s.smem < part) s.smem = part;
  }
  s.parts = n * s.cluster;
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
  p->keep = s.keep;
}

cudaError_t launch_group(const void* tile, const void* unit, GroupNormParams* p,
                         const GroupShape& s, cudaStream_t st) {
  fill_shape(p, s);
  void* args[] = {p};
  const void* fn = s.tile ? tile : unit;
  cudaError_t e = ensure_smem_attr(fn, s.smem);
  if (e == cudaSuccess && s.cluster > 8)
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  const int64_t blocks = static_cast<int64_t>(s.slabs) * p->t *
                         (s.tile ? s.parts : p->n * s.cluster);
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(fn, dim3(static_cast<unsigned>(blocks)), dim3(s.threads), s.smem, args, st,
                    s.cluster);
}

template <int DT>
static cudaError_t run_fwd(GroupNormParams* p, cudaStream_t st, int dtype) {
  const GroupShape s = group_norm_shape(p->n, p->l, p->c, p->groups, p->t, dtype, false);
  const void* tile = s.shuffle ? reinterpret_cast<const void*>(&group_tile_fwd_kernel<DT, true>)
                               : reinterpret_cast<const void*>(&group_tile_fwd_kernel<DT, false>);
  return launch_group(tile, reinterpret_cast<const void*>(&group_unit_fwd_kernel<DT>), p, s, st);
}

cudaError_t launch_group_norm_fwd(GroupNormParams p, int dtype, cudaStream_t st) {
  if (dtype == SP_BF16) return run_fwd<SP_BF16>(&p, st, dtype);
  if (dtype == SP_F16) return run_fwd<SP_F16>(&p, st, dtype);
  return run_fwd<SP_F32>(&p, st, dtype);
}

}  // namespace spb
