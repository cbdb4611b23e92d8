// Host side of the state space layer's operators (causal convolution, selective
// scan): argument validation and launch parameters.  Nothing here allocates device
// memory.
#include "region.h"
#include "region_checks.h"

using namespace spb;

namespace {

constexpr int64_t kMostBlocks = 0x7FFFFFFF;

sp_status_t check_channels(int64_t b, int64_t c) {
  if (c < 8 || c % 8 != 0)
    return fail(SP_ERR_INVALID_ARG, "c = %lld must be a positive multiple of 8", (long long)c);
  if (c > SP_MAX_HIDDEN)
    return fail(SP_ERR_UNSUPPORTED, "c = %lld above SP_MAX_HIDDEN = %d", (long long)c,
                SP_MAX_HIDDEN);
  if (b > 0xFFFFF)
    return fail(SP_ERR_UNSUPPORTED, "b = %lld above %d", (long long)b, 0xFFFFF);
  return SP_OK;
}

// Tokens find their sequence by halving, in 32 bits: the sum of two bounds has to fit.
sp_status_t check_count(const int32_t* cu_seqlens, int32_t n_seqs) {
  constexpr int32_t kMostSeqs = 1 << 30;
  if (cu_seqlens != nullptr && n_seqs > kMostSeqs)
    return fail(SP_ERR_UNSUPPORTED, "n_seqs = %d above %d", n_seqs, kMostSeqs);
  return SP_OK;
}

// Without a token every state (or gradient of one) passes through.
sp_status_t pass_states(const void* const* src, void* const* dst, size_t bytes, int t,
                        void* stream) {
  if (dst == nullptr) return SP_OK;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  for (int r = 0; r < t && bytes > 0; ++r) {
    if (src != nullptr && src[r] == dst[r]) continue;
    const cudaError_t e =
        src != nullptr ? cudaMemcpyAsync(dst[r], src[r], bytes, cudaMemcpyDeviceToDevice, cs)
                       : cudaMemsetAsync(dst[r], 0, bytes, cs);
    if (e != cudaSuccess) return fail_cuda(e, "states of no token");
  }
  return SP_OK;
}

// A parameter's gradient without a token: exact zeros.
sp_status_t zero_params(float* p, size_t count, void* stream) {
  if (p == nullptr) return SP_OK;
  const cudaError_t e = cudaMemsetAsync(p, 0, count * 4, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SP_OK : fail_cuda(e, "gradients of no token");
}

sp_status_t check_param(const void* p, bool needed, const char* what) {
  if (p == nullptr)
    return needed ? fail(SP_ERR_INVALID_ARG, "%s is NULL", what) : SP_OK;
  if (!aligned16(p)) return fail(SP_ERR_MISALIGNED, "%s misaligned", what);
  return SP_OK;
}

sp_status_t check_workspace(const void* workspace, size_t have, size_t need) {
  if (need == 0) return SP_OK;
  if (workspace == nullptr || have < need)
    return fail(SP_ERR_INVALID_ARG, "workspace of %zu bytes needed (got %zu)", need,
                workspace == nullptr ? (size_t)0 : have);
  if (!aligned16(workspace)) return fail(SP_ERR_MISALIGNED, "workspace misaligned");
  return SP_OK;
}

// ------------------------------------------------------- causal convolution --
sp_status_t check_conv(int64_t b, int64_t s, int64_t c, int32_t width, int32_t t,
                       sp_dtype_t dtype, const int32_t* cu_seqlens, int32_t n_seqs,
                       const int32_t* dev_status) {
  sp_status_t st;
  if ((st = check_common(t, dtype, dev_status)) != SP_OK) return st;
  if ((st = check_seqs(b, s, cu_seqlens, n_seqs)) != SP_OK) return st;
  if ((st = check_count(cu_seqlens, n_seqs)) != SP_OK) return st;
  if ((st = check_channels(b, c)) != SP_OK) return st;
  if (width < 2 || width > 4)
    return fail(SP_ERR_UNSUPPORTED, "width = %d outside [2, 4]", width);
  if (b * s > kMostBlocks / t / (c / 4) * 256)
    return fail(SP_ERR_UNSUPPORTED, "b * s = %lld tokens are too many", (long long)(b * s));
  return SP_OK;
}

void fill_conv(ConvParams* P, const void* const* x, int64_t x_ld, const void* weight,
               const void* bias, const void* const* x0, int64_t b, int64_t s, int64_t c,
               int32_t width, int32_t t, sp_dtype_t dtype, sp_act_t act, const int32_t* cu_seqlens,
               int32_t n_seqs, int32_t* dev_status) {
  for (int r = 0; r < t; ++r) {
    P->x[r] = static_cast<const char*>(x[r]);
    P->x0[r] = x0 != nullptr ? static_cast<const char*>(x0[r]) : nullptr;
  }
  P->ld_x = x_ld * elem_size(dtype);
  P->weight = static_cast<const char*>(weight);
  P->bias = static_cast<const char*>(bias);
  P->s = s;
  P->b = static_cast<int32_t>(b);
  P->c = static_cast<int32_t>(c);
  P->t = t;
  P->width = width;
  P->act = act;
  P->cu_seqlens = cu_seqlens;
  P->n_seqs = n_seqs;
  P->status = dev_status;
}

// ---------------------------------------------------------- selective scan --
struct Scan {
  int64_t b, s, c;
  int32_t n, groups, t;
  sp_dtype_t dtype;
  const int32_t* cu_seqlens;
  int32_t n_seqs;
  int64_t rows() const { return b * s; }
  int64_t seqs() const { return cu_seqlens != nullptr ? n_seqs : b; }
  size_t state_bytes() const { return static_cast<size_t>(seqs() * c) * n * 4; }
  size_t saved_bytes() const {
    return static_cast<size_t>(b * ((s + kSsmRun - 1) / kSsmRun)) * c * n * 4;
  }
};

sp_status_t check_scan(const Scan& k, const int32_t* dev_status) {
  sp_status_t st;
  if ((st = check_common(k.t, k.dtype, dev_status)) != SP_OK) return st;
  if ((st = check_seqs(k.b, k.s, k.cu_seqlens, k.n_seqs)) != SP_OK) return st;
  if ((st = check_count(k.cu_seqlens, k.n_seqs)) != SP_OK) return st;
  if ((st = check_channels(k.b, k.c)) != SP_OK) return st;
  if (k.n != 8 && k.n != 16 && k.n != 32 && k.n != 64)
    return fail(SP_ERR_UNSUPPORTED, "n = %d states: 8, 16, 32 or 64", k.n);
  if (k.groups < 1 || k.c % k.groups != 0 || (k.c / k.groups) % 8 != 0)
    return fail(SP_ERR_INVALID_ARG,
                "c = %lld in %d groups: whole groups of a multiple of 8 channels", (long long)k.c,
                k.groups);
  // (blocks of eight channels at least, and of 256 tokens where there are many)
  if (k.b * (k.s / 256 + 1) > kMostBlocks / k.t / (k.c / 8) / 4)
    return fail(SP_ERR_UNSUPPORTED, "b = %lld rows of s = %lld tokens are too many",
                (long long)k.b, (long long)k.s);
  return SP_OK;
}

// One tensor of a scan's call.
struct Rows {
  const void* const* p;
  int64_t ld, width;
  bool out;
  const char* what;
};

sp_status_t check_rows(const Rows& x, const Scan& k, Ranges* rg) {
  sp_status_t st;
  if ((st = check_ranks(x.p, k.t, x.what)) != SP_OK) return st;
  const int size = elem_size(k.dtype);
  for (int r = 0; r < k.t; ++r)
    rg->add_rows(x.p[r], k.rows(), x.ld * size, x.width * size, x.out, x.what, r);
  return SP_OK;
}

sp_status_t check_strides(const Rows* x, int count, const Scan& k) {
  for (int i = 0; i < count; ++i) {
    if (x[i].p == nullptr) continue;
    const sp_status_t st = check_ld(x[i].ld, x[i].width, k.rows(), x[i].what);
    if (st != SP_OK) return st;
  }
  return SP_OK;
}

void fill_scan(SsmParams* P, const Scan& k, const void* const* u, int64_t u_ld,
               const void* const* dt, int64_t dt_ld, const float* A, const void* const* B,
               int64_t B_ld, const void* const* C, int64_t C_ld, const float* D,
               const void* const* z, int64_t z_ld, const float* dt_bias, int32_t softplus,
               const float* const* h0, int32_t* dev_status) {
  const int size = elem_size(k.dtype);
  for (int r = 0; r < k.t; ++r) {
    P->u[r] = static_cast<const char*>(u[r]);
    P->dt[r] = static_cast<const char*>(dt[r]);
    P->B[r] = static_cast<const char*>(B[r]);
    P->C[r] = static_cast<const char*>(C[r]);
    P->z[r] = z != nullptr ? static_cast<const char*>(z[r]) : nullptr;
    P->h0[r] = h0 != nullptr ? h0[r] : nullptr;
  }
  P->ld_u = u_ld * size;
  P->ld_dt = dt_ld * size;
  P->ld_B = B_ld * size;
  P->ld_C = C_ld * size;
  P->ld_z = z_ld * size;
  P->A = A;
  P->D = D;
  P->dt_bias = dt_bias;
  P->s = k.s;
  P->b = static_cast<int32_t>(k.b);
  P->c = static_cast<int32_t>(k.c);
  P->t = k.t;
  P->n = k.n;
  P->groups = k.groups;
  P->softplus = softplus != 0;
  P->gated = z != nullptr;
  P->cu_seqlens = k.cu_seqlens;
  P->n_seqs = k.n_seqs;
  P->status = dev_status;
}

void put_split(SsmParams* P, const SsmSplit& split, void* workspace) {
  P->slabs = split.slabs;
  P->chunks = split.chunks;
  P->chunk_len = split.chunk_len;
  float* at = static_cast<float*>(workspace);
  P->carry = at;
  at += split.carry;
  P->steps = at;
  at += split.steps;
  P->partial_bc = split.partial_bc > 0 ? at : nullptr;
  at += split.partial_bc;
  P->partial_params = split.partial_params > 0 ? at : nullptr;
}

size_t scan_workspace(int64_t b, int64_t s, int64_t c, int32_t n, int32_t groups, int32_t t,
                      bool bwd) {
  const Scan k{b, s, c, n, groups, t, SP_F32, nullptr, 0};
  if (check_scan(k, nullptr) != SP_OK || k.rows() == 0) return 0;
  return ssm_split(b, s, c, n, groups, t, bwd).bytes();
}

}  // namespace

extern "C" {

sp_status_t sp_causal_conv_fwd(const void* const* x, int64_t x_ld, const void* weight,
                               const void* bias, const void* const* x0, int64_t b, int64_t s,
                               int64_t c, int32_t width, int32_t t, sp_dtype_t dtype, sp_act_t act,
                               const int32_t* cu_seqlens, int32_t n_seqs, void* const* y,
                               int64_t y_ld, void* const* xT, int32_t* dev_status, void* stream) {
  sp_status_t st;
  if (take_injected(&st)) return st;
  if ((st = check_conv(b, s, c, width, t, dtype, cu_seqlens, n_seqs, dev_status)) != SP_OK)
    return st;
  if (act != SP_ACT_NONE && act != SP_ACT_SILU)
    return fail(SP_ERR_INVALID_ARG, "unknown activation %d", (int)act);
  const int64_t rows = b * s, seqs = cu_seqlens != nullptr ? n_seqs : b;
  if ((st = check_ld(x_ld, c, rows, "x_ld")) != SP_OK) return st;
  if ((st = check_ld(y_ld, c, rows, "y_ld")) != SP_OK) return st;
  if (b == 0) return SP_OK;
  if (x0 != nullptr && (st = check_ranks(x0, t, "x0")) != SP_OK) return st;
  if (xT != nullptr && (st = check_ranks(xT, t, "xT")) != SP_OK) return st;
  const int size = elem_size(dtype);
  const size_t state_bytes = static_cast<size_t>(seqs * (width - 1) * c) * size;
  Ranges rg;
  if (rows > 0) {
    if ((st = check_ranks(x, t, "x")) != SP_OK) return st;
    if ((st = check_ranks(y, t, "y")) != SP_OK) return st;
    if ((st = check_param(weight, true, "weight")) != SP_OK) return st;
    if ((st = check_param(bias, false, "bias")) != SP_OK) return st;
    for (int r = 0; r < t; ++r) {
      rg.add_rows(x[r], rows, x_ld * size, c * size, false, "x", r);
      rg.add_rows(y[r], rows, y_ld * size, c * size, true, "y", r);
    }
    rg.add(weight, static_cast<size_t>(t * c) * width * size, false, "weight", 0);
    rg.add(bias, static_cast<size_t>(t * c) * size, false, "bias", 0);
  }
  for (int r = 0; r < t; ++r) {
    if (x0 != nullptr && !(xT != nullptr && xT[r] == x0[r]))
      rg.add(x0[r], state_bytes, false, "x0", r);
    if (xT != nullptr) rg.add(xT[r], state_bytes, true, "xT", r);
  }
  if (cu_seqlens != nullptr) rg.add(cu_seqlens, (n_seqs + size_t(1)) * 4, false, "cu_seqlens", 0);
  if ((st = rg.check()) != SP_OK) return st;
  if (rows == 0) return pass_states(x0, xT, state_bytes, t, stream);

  ConvParams P{};
  fill_conv(&P, x, x_ld, weight, bias, x0, b, s, c, width, t, dtype, act, cu_seqlens, n_seqs,
            dev_status);
  for (int r = 0; r < t; ++r) {
    P.out[r] = static_cast<char*>(y[r]);
    P.xT[r] = xT != nullptr ? static_cast<char*>(xT[r]) : nullptr;
  }
  P.ld_out = y_ld * size;
  const cudaError_t e = launch_conv_fwd(P, dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SP_OK : fail_cuda(e, "sp_causal_conv_fwd launch");
}

size_t sp_causal_conv_bwd_workspace_bytes(int64_t b, int64_t s, int64_t c, int32_t width,
                                          int32_t t, sp_dtype_t dtype) {
  if (check_conv(b, s, c, width, t, dtype, nullptr, 0, nullptr) != SP_OK || b * s == 0) return 0;
  return static_cast<size_t>(conv_bwd_parts(b, s, static_cast<int>(c), t, dtype)) *
         static_cast<size_t>(t * c) * (width + 1) * sizeof(float);
}

sp_status_t sp_causal_conv_bwd(const void* const* x, int64_t x_ld, const void* weight,
                               const void* bias, const void* const* x0, const void* const* dy,
                               int64_t dy_ld, const void* const* dxT, int64_t b, int64_t s,
                               int64_t c, int32_t width, int32_t t, sp_dtype_t dtype, sp_act_t act,
                               const int32_t* cu_seqlens, int32_t n_seqs, void* const* dx,
                               int64_t dx_ld, void* const* dx0, float* dweight, float* dbias,
                               void* workspace, size_t workspace_bytes, int32_t* dev_status,
                               void* stream) {
  sp_status_t st;
  if (take_injected(&st)) return st;
  if ((st = check_conv(b, s, c, width, t, dtype, cu_seqlens, n_seqs, dev_status)) != SP_OK)
    return st;
  if (act != SP_ACT_NONE && act != SP_ACT_SILU)
    return fail(SP_ERR_INVALID_ARG, "unknown activation %d", (int)act);
  const int64_t rows = b * s, seqs = cu_seqlens != nullptr ? n_seqs : b;
  const int64_t strides[] = {x_ld, dy_ld, dx_ld};
  const char* names[] = {"x_ld", "dy_ld", "dx_ld"};
  for (int i = 0; i < 3; ++i)
    if ((st = check_ld(strides[i], c, rows, names[i])) != SP_OK) return st;
  if ((st = check_param(dweight, false, "dweight")) != SP_OK) return st;
  if ((st = check_param(dbias, false, "dbias")) != SP_OK) return st;
  const size_t channels = static_cast<size_t>(t * c);
  if (x0 != nullptr && b > 0 && (st = check_ranks(x0, t, "x0")) != SP_OK) return st;
  if (dxT != nullptr && b > 0 && (st = check_ranks(dxT, t, "dxT")) != SP_OK) return st;
  if (dx0 != nullptr && b > 0 && (st = check_ranks(dx0, t, "dx0")) != SP_OK) return st;
  const int size = elem_size(dtype);
  const size_t state_bytes = static_cast<size_t>(seqs * (width - 1) * c) * size;
  const size_t need = rows > 0 && (dweight != nullptr || dbias != nullptr)
                          ? sp_causal_conv_bwd_workspace_bytes(b, s, c, width, t, dtype)
                          : 0;
  Ranges rg;
  if (rows > 0) {
    if ((st = check_ranks(x, t, "x")) != SP_OK) return st;
    if ((st = check_ranks(dy, t, "dy")) != SP_OK) return st;
    if ((st = check_ranks(dx, t, "dx")) != SP_OK) return st;
    if ((st = check_param(weight, true, "weight")) != SP_OK) return st;
    if ((st = check_param(bias, false, "bias")) != SP_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, need)) != SP_OK) return st;
    for (int r = 0; r < t; ++r) {
      rg.add_rows(x[r], rows, x_ld * size, c * size, false, "x", r);
      rg.add_rows(dy[r], rows, dy_ld * size, c * size, false, "dy", r);
      rg.add_rows(dx[r], rows, dx_ld * size, c * size, true, "dx", r);
    }
    rg.add(weight, channels * width * size, false, "weight", 0);
    rg.add(bias, channels * size, false, "bias", 0);
    if (need > 0) rg.add(workspace, need, true, "workspace", 0);
  }
  rg.add(dweight, channels * width * 4, true, "dweight", 0);
  rg.add(dbias, channels * 4, true, "dbias", 0);
  for (int r = 0; r < t; ++r) {
    if (x0 != nullptr && b > 0) rg.add(x0[r], state_bytes, false, "x0", r);
    if (dxT != nullptr && b > 0) rg.add(dxT[r], state_bytes, false, "dxT", r);
    if (dx0 != nullptr && b > 0) rg.add(dx0[r], state_bytes, true, "dx0", r);
  }
  if (cu_seqlens != nullptr) rg.add(cu_seqlens, (n_seqs + size_t(1)) * 4, false, "cu_seqlens", 0);
  if ((st = rg.check()) != SP_OK) return st;
  if (rows == 0) {
    if ((st = zero_params(dweight, channels * width, stream)) != SP_OK) return st;
    if ((st = zero_params(dbias, channels, stream)) != SP_OK) return st;
    return b > 0 ? pass_states(dxT, dx0, state_bytes, t, stream) : SP_OK;
  }

  ConvParams P{};
  fill_conv(&P, x, x_ld, weight, bias, x0, b, s, c, width, t, dtype, act, cu_seqlens, n_seqs,
            dev_status);
  for (int r = 0; r < t; ++r) {
    P.dy[r] = static_cast<const char*>(dy[r]);
    P.out[r] = static_cast<char*>(dx[r]);
    P.dxT[r] = dxT != nullptr ? static_cast<const char*>(dxT[r]) : nullptr;
    P.xT[r] = dx0 != nullptr ? static_cast<char*>(dx0[r]) : nullptr;
  }
  P.ld_dy = dy_ld * size;
  P.ld_out = dx_ld * size;
  P.ws = need > 0 ? static_cast<float*>(workspace) : nullptr;
  const cudaError_t e =
      launch_conv_bwd(P, dtype, dweight, dbias, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SP_OK : fail_cuda(e, "sp_causal_conv_bwd launch");
}

size_t sp_selective_scan_fwd_workspace_bytes(int64_t b, int64_t s, int64_t c, int32_t n,
                                             int32_t groups, int32_t t) {
  return scan_workspace(b, s, c, n, groups, t, false);
}

size_t sp_selective_scan_bwd_workspace_bytes(int64_t b, int64_t s, int64_t c, int32_t n,
                                             int32_t groups, int32_t t) {
  return scan_workspace(b, s, c, n, groups, t, true);
}

sp_status_t sp_selective_scan_fwd(const void* const* u, int64_t u_ld, const void* const* dt,
                                  int64_t dt_ld, const float* A, const void* const* B,
                                  int64_t B_ld, const void* const* C, int64_t C_ld, const float* D,
                                  const void* const* z, int64_t z_ld, const float* dt_bias,
                                  int32_t softplus, const float* const* h0, int64_t b, int64_t s,
                                  int64_t c, int32_t n, int32_t groups, int32_t t,
                                  sp_dtype_t dtype, const int32_t* cu_seqlens, int32_t n_seqs,
                                  void* const* y, int64_t y_ld, float* const* hT,
                                  float* const* states, void* workspace, size_t workspace_bytes,
                                  int32_t* dev_status, void* stream) {
  sp_status_t st;
  if (take_injected(&st)) return st;
  const Scan k{b, s, c, n, groups, t, dtype, cu_seqlens, n_seqs};
  if ((st = check_scan(k, dev_status)) != SP_OK) return st;
  const int64_t shared = static_cast<int64_t>(groups) * n;
  const Rows rows[] = {{u, u_ld, c, false, "u"},       {dt, dt_ld, c, false, "dt"},
                       {B, B_ld, shared, false, "B"},  {C, C_ld, shared, false, "C"},
                       {y, y_ld, c, true, "y"},        {z, z_ld, c, false, "z"}};
  const int count = z != nullptr ? 6 : 5;
  if ((st = check_strides(rows, count, k)) != SP_OK) return st;
  if (b == 0) return SP_OK;
  if (h0 != nullptr && (st = check_ranks(h0, t, "h0")) != SP_OK) return st;
  if (hT != nullptr && (st = check_ranks(hT, t, "hT")) != SP_OK) return st;
  Ranges rg;
  SsmSplit split{};
  bool in_place = false;
  const size_t channels = static_cast<size_t>(t * c);
  if (k.rows() > 0) {
    for (int i = 0; i < count; ++i)
      if ((st = check_rows(rows[i], k, &rg)) != SP_OK) return st;
    if (states != nullptr && (st = check_ranks(states, t, "states")) != SP_OK) return st;
    if ((st = check_param(A, true, "A")) != SP_OK) return st;
    if ((st = check_param(D, false, "D")) != SP_OK) return st;
    if ((st = check_param(dt_bias, false, "dt_bias")) != SP_OK) return st;
    split = ssm_split(b, s, c, n, groups, t, false);
    if ((st = check_workspace(workspace, workspace_bytes, split.bytes())) != SP_OK) return st;
    rg.add(A, channels * n * 4, false, "A", 0);
    rg.add(D, channels * 4, false, "D", 0);
    rg.add(dt_bias, channels * 4, false, "dt_bias", 0);
    if (split.bytes() > 0) rg.add(workspace, split.bytes(), true, "workspace", 0);
  }
  for (int r = 0; r < t; ++r) {
    const bool same = h0 != nullptr && hT != nullptr && hT[r] == h0[r];
    in_place = in_place || same;
    if (h0 != nullptr && !same) rg.add(h0[r], k.state_bytes(), false, "h0", r);
    if (hT != nullptr) rg.add(hT[r], k.state_bytes(), true, "hT", r);
    if (k.rows() > 0 && states != nullptr) rg.add(states[r], k.saved_bytes(), true, "states", r);
  }
  if (cu_seqlens != nullptr) rg.add(cu_seqlens, (n_seqs + size_t(1)) * 4, false, "cu_seqlens", 0);
  if ((st = rg.check()) != SP_OK) return st;
  if (k.rows() == 0)
    return pass_states(reinterpret_cast<const void* const*>(h0),
                       reinterpret_cast<void* const*>(hT), k.state_bytes(), t, stream);

  SsmParams P{};
  fill_scan(&P, k, u, u_ld, dt, dt_ld, A, B, B_ld, C, C_ld, D, z, z_ld, dt_bias, softplus, h0,
            dev_status);
  for (int r = 0; r < t; ++r) {
    P.y[r] = static_cast<char*>(y[r]);
    P.hT[r] = hT != nullptr ? hT[r] : nullptr;
    P.states[r] = states != nullptr ? states[r] : nullptr;
  }
  P.ld_y = y_ld * elem_size(dtype);
  put_split(&P, split, workspace);
  // Packed sequences whose states are updated in place: a chunk that reads a sequence's
  // first state would run beside the one that writes its last.
  if (in_place && cu_seqlens != nullptr) {
    P.chunks = 1;
    P.chunk_len = s;
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const bool step = cu_seqlens == nullptr && states == nullptr && s <= kSsmStepTokens;
  const cudaError_t e = step ? launch_ssm_step(P, dtype, cs) : launch_ssm_fwd(P, dtype, cs);
  return e == cudaSuccess ? SP_OK : fail_cuda(e, "sp_selective_scan_fwd launch");
}

sp_status_t sp_selective_scan_bwd(const void* const* u, int64_t u_ld, const void* const* dt,
                                  int64_t dt_ld, const float* A, const void* const* B,
                                  int64_t B_ld, const void* const* C, int64_t C_ld, const float* D,
                                  const void* const* z, int64_t z_ld, const float* dt_bias,
                                  int32_t softplus, const float* const* h0,
                                  const float* const* states, const void* const* dy, int64_t dy_ld,
                                  const float* const* dhT, int64_t b, int64_t s, int64_t c,
                                  int32_t n, int32_t groups, int32_t t, sp_dtype_t dtype,
                                  const int32_t* cu_seqlens, int32_t n_seqs, void* const* du,
                                  int64_t du_ld, void* const* ddt, int64_t ddt_ld, void* const* dB,
                                  int64_t dB_ld, void* const* dC, int64_t dC_ld, void* const* dz,
                                  int64_t dz_ld, float* dA, float* dD, float* ddt_bias,
                                  float* const* dh0, void* workspace, size_t workspace_bytes,
                                  int32_t* dev_status, void* stream) {
  sp_status_t st;
  if (take_injected(&st)) return st;
  const Scan k{b, s, c, n, groups, t, dtype, cu_seqlens, n_seqs};
  if ((st = check_scan(k, dev_status)) != SP_OK) return st;
  const int64_t shared = static_cast<int64_t>(groups) * n;
  const Rows rows[] = {
      {u, u_ld, c, false, "u"},       {dt, dt_ld, c, false, "dt"},   {B, B_ld, shared, false, "B"},
      {C, C_ld, shared, false, "C"},  {dy, dy_ld, c, false, "dy"},   {du, du_ld, c, true, "du"},
      {ddt, ddt_ld, c, true, "ddt"},  {dB, dB_ld, shared, true, "dB"},
      {dC, dC_ld, shared, true, "dC"}, {z, z_ld, c, false, "z"},     {dz, dz_ld, c, true, "dz"}};
  const int count = z != nullptr ? 11 : 9;
  if ((st = check_strides(rows, count, k)) != SP_OK) return st;
  struct { const float* p; size_t count; const char* what; } grads[] = {
      {dA, static_cast<size_t>(t * c) * n, "dA"},
      {dD, static_cast<size_t>(t * c), "dD"},
      {ddt_bias, static_cast<size_t>(t * c), "ddt_bias"}};
  Ranges rg;
  for (const auto& g : grads) {
    if ((st = check_param(g.p, false, g.what)) != SP_OK) return st;
    rg.add(g.p, g.count * 4, true, g.what, 0);
  }
  if (b > 0) {
    if (h0 != nullptr && (st = check_ranks(h0, t, "h0")) != SP_OK) return st;
    if (dhT != nullptr && (st = check_ranks(dhT, t, "dhT")) != SP_OK) return st;
    if (dh0 != nullptr && (st = check_ranks(dh0, t, "dh0")) != SP_OK) return st;
  }
  SsmSplit split{};
  const size_t channels = static_cast<size_t>(t * c);
  if (k.rows() > 0) {
    for (int i = 0; i < count; ++i)
      if ((st = check_rows(rows[i], k, &rg)) != SP_OK) return st;
    if ((st = check_ranks(states, t, "states")) != SP_OK) return st;
    if ((st = check_param(A, true, "A")) != SP_OK) return st;
    if ((st = check_param(D, false, "D")) != SP_OK) return st;
    if ((st = check_param(dt_bias, false, "dt_bias")) != SP_OK) return st;
    split = ssm_split(b, s, c, n, groups, t, true);
    if ((st = check_workspace(workspace, workspace_bytes, split.bytes())) != SP_OK) return st;
    rg.add(A, channels * n * 4, false, "A", 0);
    rg.add(D, channels * 4, false, "D", 0);
    rg.add(dt_bias, channels * 4, false, "dt_bias", 0);
    if (split.bytes() > 0) rg.add(workspace, split.bytes(), true, "workspace", 0);
  }
  for (int r = 0; r < t && b > 0; ++r) {
    if (k.rows() > 0) rg.add(states[r], k.saved_bytes(), false, "states", r);
    if (h0 != nullptr) rg.add(h0[r], k.state_bytes(), false, "h0", r);
    if (dhT != nullptr) rg.add(dhT[r], k.state_bytes(), false, "dhT", r);
    if (dh0 != nullptr) rg.add(dh0[r], k.state_bytes(), true, "dh0", r);
  }
  if (cu_seqlens != nullptr) rg.add(cu_seqlens, (n_seqs + size_t(1)) * 4, false, "cu_seqlens", 0);
  if ((st = rg.check()) != SP_OK) return st;
  if (k.rows() == 0) {
    if ((st = zero_params(dA, channels * n, stream)) != SP_OK) return st;
    if ((st = zero_params(dD, channels, stream)) != SP_OK) return st;
    if ((st = zero_params(ddt_bias, channels, stream)) != SP_OK) return st;
    return b > 0 ? pass_states(reinterpret_cast<const void* const*>(dhT),
                               reinterpret_cast<void* const*>(dh0), k.state_bytes(), t, stream)
                 : SP_OK;
  }

  SsmParams P{};
  fill_scan(&P, k, u, u_ld, dt, dt_ld, A, B, B_ld, C, C_ld, D, z, z_ld, dt_bias, softplus, h0,
            dev_status);
  for (int r = 0; r < t; ++r) {
    P.dy[r] = static_cast<const char*>(dy[r]);
    P.du[r] = static_cast<char*>(du[r]);
    P.ddt[r] = static_cast<char*>(ddt[r]);
    P.dB[r] = static_cast<char*>(dB[r]);
    P.dC[r] = static_cast<char*>(dC[r]);
    P.dz[r] = z != nullptr ? static_cast<char*>(dz[r]) : nullptr;
    P.states[r] = const_cast<float*>(states[r]);
    P.dhT[r] = dhT != nullptr ? dhT[r] : nullptr;
    P.hT[r] = dh0 != nullptr ? dh0[r] : nullptr;
  }
  const int size = elem_size(dtype);
  P.ld_dy = dy_ld * size;
  P.ld_du = du_ld * size;
  P.ld_ddt = ddt_ld * size;
  P.ld_dB = dB_ld * size;
  P.ld_dC = dC_ld * size;
  P.ld_dz = dz_ld * size;
  put_split(&P, split, workspace);
  if (dA == nullptr && dD == nullptr && ddt_bias == nullptr) P.partial_params = nullptr;
  const cudaError_t e = launch_ssm_bwd(P, dtype, SsmParamGrads{dA, dD, ddt_bias},
                                       static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SP_OK : fail_cuda(e, "sp_selective_scan_bwd launch");
}

}  // extern "C"
