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

constexpr int kBackTileRows = 4;    // vectors of x and dy a thread holds (tiles)
constexpr int kBackUnitBatch = 4;   // vectors of each a thread reads at once (units)

template <int DT, bool SHFL>
__global__ void __launch_bounds__(kGroupThreads) group_tile_bwd_kernel(const GroupNormParams P) {
  constexpr int E = ElemSize<DT>::value;
  extern __shared__ float2 dyn2[];             // [tile rows][cols] sums, then [pairs]
  pdl_wait();
  const int cx = threadIdx.x % P.cols, ry = threadIdx.x / P.cols;
  const int slab = blockIdx.x % P.slabs;
  const int r = blockIdx.x / P.slabs % P.t;
  const int64_t part = blockIdx.x / (P.slabs * P.t);
  const int vec = slab * P.cols + cx;
  const bool on = ry < P.rows && vec * 8 < P.c;
  const bool ln = P.norm == SP_NORM_LAYERNORM, silu = P.act == SP_ACT_SILU;
  const int64_t ch = static_cast<int64_t>(r) * P.c + vec * 8;
  Column<DT> col;
  col.read(P, ch, on);
  const int64_t at = static_cast<int64_t>(vec) * 8 * E;
  const char* x = P.x[r] + at;
  const char* dy = P.dy[r] + at;
  char* out = P.out[r] + at;
  const int tile_rows = static_cast<int>(P.samples * P.l);
  const int slab_groups = P.cols / P.q;
  const int pairs = P.samples * slab_groups;
  float2* stat = dyn2 + P.rows * kBackTileRows * P.cols;
  const int group = vec / P.q;
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;

  for (int64_t s0 = part * P.samples; s0 < P.n; s0 += P.parts * P.samples) {
    const int64_t row0 = s0 * P.l;
    const int64_t left = P.n * P.l - row0;
    const int here = left < tile_rows ? static_cast<int>(left) : tile_rows;
    Vec8<DT> xraw[kBackTileRows], draw[kBackTileRows];
    float mean[kBackTileRows], rstd[kBackTileRows];
#pragma unroll
    for (int u = 0; u < kBackTileRows; ++u) {
      xraw[u] = draw[u] = Vec8<DT>{};
      mean[u] = rstd[u] = 0.f;
      const int row = ry + u * P.rows;
      if (on && row < here) {
        load_pack(xraw[u], x + (row0 + row) * P.ld_x);
        load_pack(draw[u], dy + (row0 + row) * P.ld_dy);
        const int64_t st = (SHFL ? row0 + row : s0 + row / static_cast<int>(P.l)) * P.groups + group;
        if (ln) mean[u] = __ldg(P.mean[r] + st);
        rstd[u] = __ldg(P.rstd[r] + st);
      }
    }
    float2 sum[kBackTileRows];                 // sums of dz and of dz z
#pragma unroll
    for (int u = 0; u < kBackTileRows; ++u) {
      float f[8], d[8], z[8], dq[8];
      unpack(xraw[u], f);
      unpack(draw[u], d);
      back_act<DT>(f, d, mean[u], rstd[u], col, silu, z, dq);
      sum[u] = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[i] = fmaf(dq[i], z[i], acc[i]);
        acc[8 + i] += dq[i];
        const float dz = dq[i] * col.gamma[i];
        sum[u].x += dz;
        sum[u].y = fmaf(dz, z[i], sum[u].y);
      }
      if constexpr (SHFL) {
        sum[u].x = lanes_sum(sum[u].x, P.q);
        sum[u].y = lanes_sum(sum[u].y, P.q);
      }
    }
    if constexpr (!SHFL) {
#pragma unroll
      for (int u = 0; u < kBackTileRows; ++u)
        if (ry < P.rows) dyn2[(ry + u * P.rows) * P.cols + cx] = sum[u];
      __syncthreads();
      const int lane = threadIdx.x % P.lanes, step = blockDim.x / P.lanes;
      for (int p0 = 0; p0 < pairs; p0 += step) {
        const int p = p0 + threadIdx.x / P.lanes;
        float2 v = make_float2(0.f, 0.f);
        if (p < pairs) {
          const int s = p / slab_groups, g = p - s * slab_groups;
          const int terms = static_cast<int>(P.l) * P.q;
          for (int e = lane; e < terms; e += P.lanes) {
            const int i = e / P.q;
            const float2 w =
                dyn2[(s * static_cast<int>(P.l) + i) * P.cols + g * P.q + (e - i * P.q)];
            v.x += w.x;
            v.y += w.y;
          }
        }
        v.x = lanes_sum(v.x, P.lanes);
        v.y = lanes_sum(v.y, P.lanes);
        if (p < pairs && lane == 0) stat[p] = v;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kBackTileRows; ++u) {
        const int row = ry + u * P.rows;
        if (row < tile_rows)
          sum[u] = stat[row / static_cast<int>(P.l) * slab_groups + cx / P.q];
      }
    }
#pragma unroll
    for (int u = 0; u < kBackTileRows; ++u) {
      const int row = ry + u * P.rows;
      if (!on || row >= here) continue;
      float f[8], d[8], z[8], dq[8];
      unpack(xraw[u], f);
      unpack(draw[u], d);
      back_act<DT>(f, d, mean[u], rstd[u], col, silu, z, dq);
      const float m1 = ln ? sum[u].x * P.count_inv : 0.f, m2 = sum[u].y * P.count_inv;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        f[i] = rstd[u] * (fmaf(dq[i], col.gamma[i], -m1) - z[i] * m2);
      Vec8<DT> o;
      pack(o, f);
      store_pack(out + (row0 + row) * P.ld_out, o);
    }
    if constexpr (!SHFL) __syncthreads();
  }
  if (P.has_params)
    put_param_part(P, acc, reinterpret_cast<float*>(dyn2), cx, ry, on, ch, part);
}

template <int DT>
__global__ void __launch_bounds__(kGroupThreads) group_unit_bwd_kernel(const GroupNormParams P) {
  constexpr int E = ElemSize<DT>::value;
  extern __shared__ uint4 kept[];              // [keep][x, dy][threads] vectors, then the sums
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
  float2* sums = reinterpret_cast<float2*>(kept + static_cast<int64_t>(P.keep) * 2 * kPer *
                                                      blockDim.x);
  float2* joined = sums + blockDim.x;          // [cluster][slab groups] sums of each block
  float2* stat = joined + C * slab_groups;     // [slab groups] group means of dz and dz z
  const int64_t ch = static_cast<int64_t>(r) * P.c + vec * 8;
  Column<DT> col;
  col.read(P, ch, on);
  const int64_t b0 = P.l * rank / C, b1 = P.l * (rank + 1) / C;
  const int mine =
      on && b1 - b0 > ry ? static_cast<int>((b1 - b0 - ry + P.rows - 1) / P.rows) : 0;
  const int64_t row0 = sample * P.l + b0 + ry;
  const int64_t at = static_cast<int64_t>(vec) * 8 * E;
  const char* x = P.x[r] + row0 * P.ld_x + at;
  const char* dy = P.dy[r] + row0 * P.ld_dy + at;
  char* out = P.out[r] + row0 * P.ld_out + at;
  const int64_t step_x = P.ld_x * P.rows, step_dy = P.ld_dy * P.rows, step_out = P.ld_out * P.rows;
  float mean = 0.f, rstd = 0.f;
  if (on) {
    const int64_t g = sample * P.groups + vec / P.q;
    if (ln) mean = __ldg(P.mean[r] + g);
    rstd = __ldg(P.rstd[r] + g);
  }
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int i0 = 0; i0 < mine; i0 += kBackUnitBatch) {
    Vec8<DT> xraw[kBackUnitBatch], draw[kBackUnitBatch];
#pragma unroll
    for (int u = 0; u < kBackUnitBatch; ++u) {
      xraw[u] = draw[u] = Vec8<DT>{};
      if (i0 + u < mine) {
        load_pack(xraw[u], x + (i0 + u) * step_x);
        load_pack(draw[u], dy + (i0 + u) * step_dy);
      }
    }
#pragma unroll
    for (int u = 0; u < kBackUnitBatch; ++u) {
      if (i0 + u >= mine) continue;
      if (i0 + u < P.keep) {
        uint4* to = kept + static_cast<int64_t>(i0 + u) * 2 * kPer * blockDim.x + threadIdx.x;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          to[k * blockDim.x] = make_uint4(xraw[u].w[4 * k], xraw[u].w[4 * k + 1],
                                          xraw[u].w[4 * k + 2], xraw[u].w[4 * k + 3]);
          to[(kPer + k) * blockDim.x] = make_uint4(draw[u].w[4 * k], draw[u].w[4 * k + 1],
                                                   draw[u].w[4 * k + 2], draw[u].w[4 * k + 3]);
        }
      }
      float f[8], d[8], z[8], dq[8];
      unpack(xraw[u], f);
      unpack(draw[u], d);
      back_act<DT>(f, d, mean, rstd, col, silu, z, dq);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[i] = fmaf(dq[i], z[i], acc[i]);
        acc[8 + i] += dq[i];
      }
    }
  }
  float2 own = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    own.x = fmaf(col.gamma[i], acc[8 + i], own.x);
    own.y = fmaf(col.gamma[i], acc[i], own.y);
  }
  if (ry < P.rows) sums[threadIdx.x] = own;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int terms = P.rows * P.q;
  for (int g = warp; g < slab_groups; g += nw) {
    float2 v = make_float2(0.f, 0.f);
    for (int e = lane; e < terms; e += 32) {
      const int y = e / P.q;
      const float2 w = sums[y * P.cols + g * P.q + (e - y * P.q)];
      v.x += w.x;
      v.y += w.y;
    }
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if (C == 1) {
      if (lane == 0) joined[g] = v;
    } else if (lane < C) {
      const uint32_t to = cluster_map(&joined[rank * slab_groups + g], lane);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(v.x), "f"(v.y)
                   : "memory");
    }
  }
  if (C > 1) cluster_sync_all(); else __syncthreads();
  for (int g = threadIdx.x; g < slab_groups; g += blockDim.x) {
    float2 v = make_float2(0.f, 0.f);
    for (int k = 0; k < C; ++k) {
      v.x += joined[k * slab_groups + g].x;
      v.y += joined[k * slab_groups + g].y;
    }
    stat[g] = make_float2(ln ? v.x * P.count_inv : 0.f, v.y * P.count_inv);
  }
  __syncthreads();
  const float2 m = stat[cx / P.q];
  for (int i0 = 0; i0 < mine; i0 += kBackUnitBatch) {
    Vec8<DT> xraw[kBackUnitBatch], draw[kBackUnitBatch];
#pragma unroll
    for (int u = 0; u < kBackUnitBatch; ++u) {
      const int i = i0 + u;
      if (i >= mine) continue;
      if (i < P.keep) {
        const uint4* from = kept + static_cast<int64_t>(i) * 2 * kPer * blockDim.x + threadIdx.x;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const uint4 v = from[k * blockDim.x], w = from[(kPer + k) * blockDim.x];
          xraw[u].w[4 * k] = v.x;
          xraw[u].w[4 * k + 1] = v.y;
          xraw[u].w[4 * k + 2] = v.z;
          xraw[u].w[4 * k + 3] = v.w;
          draw[u].w[4 * k] = w.x;
          draw[u].w[4 * k + 1] = w.y;
          draw[u].w[4 * k + 2] = w.z;
          draw[u].w[4 * k + 3] = w.w;
        }
      } else {
        load_pack(xraw[u], x + i * step_x);
        load_pack(draw[u], dy + i * step_dy);
      }
    }
#pragma unroll
    for (int u = 0; u < kBackUnitBatch; ++u) {
      if (i0 + u >= mine) continue;
      float f[8], d[8], z[8], dq[8];
      unpack(xraw[u], f);
      unpack(draw[u], d);
      back_act<DT>(f, d, mean, rstd, col, silu, z, dq);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        f[i] = rstd * (fmaf(dq[i], col.gamma[i], -m.x) - z[i] * m.y);
      Vec8<DT> o;
      pack(o, f);
      store_pack(out + (i0 + u) * step_out, o);
    }
  }
  if (P.has_params)
    put_param_part(P, acc, reinterpret_cast<float*>(kept), cx, ry, on, ch, sample * C + rank);
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
static cudaError_t run_bwd(GroupNormParams* p, cudaStream_t st, int dtype) {
  const GroupShape s = group_norm_shape(p->n, p->l, p->c, p->groups, p->t, dtype, true);
  const void* tile = s.shuffle ? reinterpret_cast<const void*>(&group_tile_bwd_kernel<DT, true>)
                               : reinterpret_cast<const void*>(&group_tile_bwd_kernel<DT, false>);
  return launch_group(tile, reinterpret_cast<const void*>(&group_unit_bwd_kernel<DT>), p, s, st);
}

cudaError_t launch_group_norm_bwd(GroupNormParams p, int dtype, float* dgamma, float* dbeta,
                                  cudaStream_t st) {
  p.has_params = dgamma != nullptr || dbeta != nullptr;
  cudaError_t e = dtype == SP_BF16  ? run_bwd<SP_BF16>(&p, st, dtype)
                  : dtype == SP_F16 ? run_bwd<SP_F16>(&p, st, dtype)
                                    : run_bwd<SP_F32>(&p, st, dtype);
  if (e != cudaSuccess || !p.has_params) return e;
  const float* ws = p.ws;
  int64_t parts = p.parts, width = static_cast<int64_t>(p.t) * p.c;
  void* args[] = {&ws, &parts, &width, &dgamma, &dbeta};
  return launch_pdl(reinterpret_cast<const void*>(&group_params_kernel),
                    dim3(static_cast<unsigned>((width + 31) / 32), 2), dim3(256), 0, args, st);
}

}  // namespace spb
