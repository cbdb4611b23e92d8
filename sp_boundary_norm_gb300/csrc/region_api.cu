// Host side of the operators between g and the next g*: argument validation
// and launch parameters.  Nothing here allocates device memory.
#include <cmath>

#include "region.h"
#include "region_checks.h"

using namespace spb;

namespace {

// ------------------------------------------------------------------ rotary --
// What a table says: of one position a token, or (axis != NULL) of a coordinate for
// each of several axes.
struct RopeTurns {
  int32_t pairs;
  float mscale;
  const uint64_t* turns;
  const uint8_t* axis;
  int32_t axes;
};

sp_status_t read_table(const sp_rope_table_t* table, RopeTurns* out) {
  if (table == nullptr) return fail(SP_ERR_INVALID_ARG, "table is NULL");
  if (table->pairs < 1 || table->pairs > SP_ROPE_MAX_PAIRS)
    return fail(SP_ERR_INVALID_ARG, "table with %d pairs: fill it with sp_rope_table",
                table->pairs);
  *out = RopeTurns{table->pairs, table->mscale, table->turns, nullptr, 1};
  return SP_OK;
}

sp_status_t read_table(const sp_rope_axes_table_t* table, RopeTurns* out) {
  if (table == nullptr) return fail(SP_ERR_INVALID_ARG, "table is NULL");
  bool good = table->pairs >= 1 && table->pairs <= SP_ROPE_MAX_PAIRS && table->axes >= 1 &&
              table->axes <= SP_ROPE_MAX_AXES;
  for (int i = 0; good && i < table->pairs; ++i) good = table->axis[i] < table->axes;
  if (!good)
    return fail(SP_ERR_INVALID_ARG, "table of %d pairs and %d axes: fill it with "
                "sp_rope_axes_table", table->pairs, table->axes);
  *out = RopeTurns{table->pairs, table->mscale, table->turns, table->axis, table->axes};
  return SP_OK;
}

template <typename Table>
sp_status_t rope(const void* const* x, int64_t x_ld, int64_t x_head, int64_t b, int64_t s,
                 int64_t heads, int64_t d, int32_t t, sp_dtype_t dtype,
                 const Table* table, sp_rope_layout_t layout, const int64_t* positions,
                 int64_t first, const int32_t* cu_seqlens, int32_t n_seqs, void* const* y,
                 int64_t y_ld, int64_t y_head, int32_t* dev_status, void* stream, float sign) {
  sp_status_t st;
  if (take_injected(&st)) return st;
  if ((st = check_common(t, dtype, dev_status)) != SP_OK) return st;
  if ((st = check_seqs(b, s, cu_seqlens, n_seqs)) != SP_OK) return st;
  if (layout != SP_ROPE_HALF && layout != SP_ROPE_INTERLEAVED)
    return fail(SP_ERR_INVALID_ARG, "unknown layout %d", (int)layout);
  RopeTurns turns;
  if ((st = read_table(table, &turns)) != SP_OK) return st;
  if (heads < 1 || heads > SP_ROPE_MAX_HEADS)
    return fail(SP_ERR_INVALID_ARG, "heads = %lld outside [1, %d]", (long long)heads,
                SP_ROPE_MAX_HEADS);
  const int64_t rot = 2 * static_cast<int64_t>(turns.pairs);
  if (d < rot || d > SP_MAX_HIDDEN)
    return fail(SP_ERR_INVALID_ARG, "d = %lld outside [rot_dim = %lld, %d]", (long long)d,
                (long long)rot, SP_MAX_HIDDEN);
  if (positions != nullptr && cu_seqlens != nullptr)
    return fail(SP_ERR_INVALID_ARG, "positions and cu_seqlens exclude each other");
  if (reinterpret_cast<uintptr_t>(positions) & 7u)
    return fail(SP_ERR_MISALIGNED, "positions not 8-byte aligned");
  const int64_t tokens = b * s;
  for (int k = 0; k < 2; ++k) {
    const int64_t head = k ? y_head : x_head, ld = k ? y_ld : x_ld;
    if (head < d || head > kMostElements || ld > kMostElements || ld < (heads - 1) * head + d)
      return fail(SP_ERR_INVALID_ARG, "%s strides: %lld between heads of %lld, %lld between tokens",
                  k ? "output" : "input", (long long)head, (long long)d, (long long)ld);
    if (tokens > 0 && ld > kMostElements / tokens)
      return fail(SP_ERR_INVALID_ARG, "the tensor's extent overflows");
  }
  if (tokens == 0) return SP_OK;
  if (turns.axis != nullptr && positions == nullptr)
    return fail(SP_ERR_INVALID_ARG, "positions is NULL");
  if ((st = check_ranks(x, t, "x")) != SP_OK) return st;
  if ((st = check_ranks(y, t, "y")) != SP_OK) return st;
  const int size = elem_size(dtype);
  const bool same_strides = x_ld == y_ld && x_head == y_head;
  bool in_place = same_strides;
  Ranges rg;
  for (int r = 0; r < t; ++r) {
    const size_t xw = ((heads - 1) * x_head + d) * size, yw = ((heads - 1) * y_head + d) * size;
    const bool here = same_strides && x[r] == y[r];
    in_place = in_place && here;
    if (!here) rg.add_rows(x[r], tokens, x_ld * size, xw, false, "x", r);
    rg.add_rows(y[r], tokens, y_ld * size, yw, true, "y", r);
  }
  if (positions != nullptr) rg.add(positions, tokens * 8 * turns.axes, false, "positions", 0);
  if (cu_seqlens != nullptr) rg.add(cu_seqlens, (n_seqs + size_t(1)) * 4, false, "cu_seqlens", 0);
  if ((st = rg.check()) != SP_OK) return st;

  // the widest accesses that the sizes and strides allow
  const int64_t block = layout == SP_ROPE_HALF ? turns.pairs : rot;
  int vec = 16 / size;
  while (vec > 1 && (block % vec != 0 || x_ld % vec != 0 || x_head % vec != 0 ||
                     y_ld % vec != 0 || y_head % vec != 0))
    vec /= 2;

  RopeAxesParams P{};
  for (int r = 0; r < t; ++r) {
    P.x[r] = static_cast<const char*>(x[r]);
    P.y[r] = static_cast<char*>(y[r]);
  }
  P.x_row = x_ld * size;
  P.x_head = x_head * size;
  P.y_row = y_ld * size;
  P.y_head = y_head * size;
  P.s = s;
  P.tokens = tokens;
  P.heads = static_cast<int32_t>(heads);
  P.all_heads = static_cast<int32_t>(heads * t);
  P.heads_magic = heads == 1 ? 0u
                             : static_cast<uint32_t>(((uint64_t(1) << 32) + heads - 1) / heads);
  P.half = turns.pairs;
  P.rest_at = static_cast<int32_t>(rot) * size;
  P.rest = in_place ? 0 : static_cast<int32_t>(d - rot) * size;
  P.rest_bytes = 16;
  while (P.rest_bytes > size && (P.rest_at % P.rest_bytes != 0 || P.rest % P.rest_bytes != 0 ||
                                 P.x_row % P.rest_bytes != 0 || P.x_head % P.rest_bytes != 0 ||
                                 P.y_row % P.rest_bytes != 0 || P.y_head % P.rest_bytes != 0))
    P.rest_bytes /= 2;
  P.layout = layout;
  P.positions = positions;
  P.first = first;
  P.cu_seqlens = cu_seqlens;
  P.n_seqs = n_seqs;
  P.cos_scale = turns.mscale;
  P.sin_scale = sign * turns.mscale;
  P.status = dev_status;
  for (int i = 0; i < turns.pairs; ++i) P.turns[i] = turns.turns[i];
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (turns.axis != nullptr)
    for (int i = 0; i < turns.pairs; ++i) P.axis[i] = turns.axis[i];
  const cudaError_t e = turns.axis != nullptr ? launch_rope_axes(P, dtype, vec, cs)
                                              : launch_rope(P, dtype, vec, cs);
  return e == cudaSuccess ? SP_OK : fail_cuda(e, "rotary launch");
}

// ---------------------------------------------------------- gated recurrence --
struct ScanCall {
  int64_t b, s, c;
  int32_t t;
  sp_dtype_t dtype;
  const int32_t* cu_seqlens;
  int32_t n_seqs;
  int64_t seqs() const { return cu_seqlens != nullptr ? n_seqs : b; }
};

sp_status_t check_scan(const ScanCall& k, const int32_t* dev_status) {
  sp_status_t st;
  if ((st = check_common(k.t, k.dtype, dev_status)) != SP_OK) return st;
  if ((st = check_seqs(k.b, k.s, k.cu_seqlens, k.n_seqs)) != SP_OK) return st;
  if (k.c < 8 || k.c % 8 != 0)
    return fail(SP_ERR_INVALID_ARG, "c = %lld must be a positive multiple of 8", (long long)k.c);
  if (k.c > SP_MAX_HIDDEN)
    return fail(SP_ERR_UNSUPPORTED, "c = %lld above SP_MAX_HIDDEN = %d", (long long)k.c,
                SP_MAX_HIDDEN);
  if (k.b > 0xFFFFF)
    return fail(SP_ERR_UNSUPPORTED, "b = %lld above %d", (long long)k.b, 0xFFFFF);
  return SP_OK;
}

// Without a token every state (or gradient of one) passes through.
sp_status_t pass_states(const ScanCall& k, const float* const* src, float* const* dst,
                        void* stream) {
  if (dst == nullptr) return SP_OK;
  const size_t bytes = static_cast<size_t>(k.seqs() * k.c) * 4;
  for (int r = 0; r < k.t && bytes > 0; ++r) {
    if (src != nullptr && src[r] == dst[r]) continue;
    const cudaError_t e =
        src != nullptr ? cudaMemcpyAsync(dst[r], src[r], bytes, cudaMemcpyDeviceToDevice,
                                         static_cast<cudaStream_t>(stream))
                       : cudaMemsetAsync(dst[r], 0, bytes, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail_cuda(e, "gated scan of no token");
  }
  return SP_OK;
}

void fill_scan(ScanParams* P, const ScanCall& k, const void* const* gate, int64_t gate_ld,
               const void* const* value, int64_t value_ld, const float* const* h0, int32_t tied,
               int32_t* dev_status) {
  const int size = elem_size(k.dtype);
  for (int r = 0; r < k.t; ++r) {
    P->gate[r] = static_cast<const char*>(gate[r]);
    P->value[r] = static_cast<const char*>(value[r]);
    P->h0[r] = h0 != nullptr ? h0[r] : nullptr;
  }
  P->ld_gate = static_cast<uint32_t>(gate_ld * size);
  P->ld_value = static_cast<uint32_t>(value_ld * size);
  P->s = k.s;
  P->b = static_cast<int32_t>(k.b);
  P->c = static_cast<int32_t>(k.c);
  P->t = k.t;
  P->slabs = static_cast<int32_t>((k.c + kScanChannels - 1) / kScanChannels);
  P->tied = tied != 0;
  P->cu_seqlens = k.cu_seqlens;
  P->n_seqs = k.n_seqs;
  P->status = dev_status;
  P->withhold = take_withheld_step();
}

// ---------------------------------------------------------------- group norm --
sp_status_t check_group(int64_t n, int64_t l, int64_t c, int64_t groups, int32_t t,
                        sp_dtype_t dtype) {
  sp_status_t st;
  if ((st = check_common(t, dtype, nullptr)) != SP_OK) return st;
  if (n < 0 || l < 0) return fail(SP_ERR_INVALID_ARG, "negative n or l");
  if (n > kMostElements || l > kMostElements || (l > 0 && n > kMostElements / l))
    return fail(SP_ERR_INVALID_ARG, "n*l overflows");
  if (c < 8 || c > SP_MAX_HIDDEN || groups < 1 || groups > c || c % groups != 0 ||
      (c / groups) % 8 != 0)
    return fail(SP_ERR_INVALID_ARG,
                "c = %lld in %lld groups: whole groups of a multiple of 8 channels, c <= %d",
                (long long)c, (long long)groups, SP_MAX_HIDDEN);
  if (c / groups > SP_MAX_GROUP_CHANNELS)
    return fail(SP_ERR_UNSUPPORTED, "groups of %lld channels above SP_MAX_GROUP_CHANNELS = %d",
                (long long)(c / groups), SP_MAX_GROUP_CHANNELS);
  if (l > 0x7FFFFFFF / 16)
    return fail(SP_ERR_UNSUPPORTED, "l = %lld rows a sample above %d", (long long)l,
                0x7FFFFFFF / 16);
  return SP_OK;
}

sp_status_t check_param(const void* p, const char* what) {
  if (p == nullptr) return fail(SP_ERR_INVALID_ARG, "%s is NULL", what);
  if (!aligned16(p)) return fail(SP_ERR_MISALIGNED, "%s misaligned", what);
  return SP_OK;
}

// Statistics are read and written one float at a time: 4-byte alignment.
sp_status_t check_stats(float* const* arr, int t, const char* what) {
  if (arr == nullptr) return fail(SP_ERR_INVALID_ARG, "%s array is NULL", what);
  for (int i = 0; i < t; ++i) {
    if (arr[i] == nullptr) return fail(SP_ERR_INVALID_ARG, "%s[%d] is NULL", what, i);
    if (reinterpret_cast<uintptr_t>(arr[i]) & 3u)
      return fail(SP_ERR_MISALIGNED, "%s[%d] misaligned", what, i);
  }
  return SP_OK;
}

sp_status_t check_act(sp_norm_t norm, sp_act_t act) {
  if (norm != SP_NORM_LAYERNORM && norm != SP_NORM_RMSNORM)
    return fail(SP_ERR_INVALID_ARG, "unknown norm %d", (int)norm);
  if (act != SP_ACT_NONE && act != SP_ACT_SILU)
    return fail(SP_ERR_INVALID_ARG, "unknown activation %d", (int)act);
  return SP_OK;
}

void fill_group(GroupNormParams* P, int64_t n, int64_t l, int64_t c, int64_t groups, int32_t t,
                sp_norm_t norm, sp_act_t act, const void* gamma, const void* beta) {
  P->n = n;
  P->l = l;
  P->c = static_cast<int32_t>(c);
  P->t = t;
  P->groups = static_cast<int32_t>(groups);
  P->norm = norm;
  P->act = act;
  P->gamma = static_cast<const char*>(gamma);
  P->beta = static_cast<const char*>(beta);
  const double count = static_cast<double>(l) * static_cast<double>(c / groups);
  P->count = static_cast<float>(count);
  P->count_inv = static_cast<float>(1.0 / count);
}

}  // namespace

extern "C" {

sp_status_t sp_rope_table(int32_t rot_dim, double base, sp_rope_scaling_t scaling, double factor,
                          int64_t original_len, double low_turns, double high_turns, double mscale,
                          sp_rope_table_t* out) {
  if (out == nullptr) return fail(SP_ERR_INVALID_ARG, "out is NULL");
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 2 * SP_ROPE_MAX_PAIRS)
    return fail(SP_ERR_INVALID_ARG, "rot_dim = %d must be even, 2 .. %d", rot_dim,
                2 * SP_ROPE_MAX_PAIRS);
  if (!(base >= 1.0) || !std::isfinite(base)) return fail(SP_ERR_INVALID_ARG, "base must be >= 1");
  if (scaling < SP_ROPE_PLAIN || scaling > SP_ROPE_PARTS)
    return fail(SP_ERR_INVALID_ARG, "unknown scaling %d", (int)scaling);
  if (!std::isfinite(mscale)) return fail(SP_ERR_INVALID_ARG, "mscale must be finite");
  if (scaling != SP_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(SP_ERR_INVALID_ARG, "factor must be >= 1");
  if (scaling == SP_ROPE_BASE && rot_dim == 2)
    return fail(SP_ERR_INVALID_ARG, "scaling the base needs rot_dim > 2");
  if (scaling == SP_ROPE_PARTS &&
      (original_len < 1 || !(high_turns > low_turns) || !std::isfinite(high_turns - low_turns)))
    return fail(SP_ERR_INVALID_ARG, "scaling by parts needs original_len > 0 and "
                "high_turns > low_turns");
  const double kTau = 6.283185307179586476925286766559;
  const double dim = rot_dim;
  const double b = scaling == SP_ROPE_BASE ? base * std::pow(factor, dim / (dim - 2)) : base;
  if (!std::isfinite(b)) return fail(SP_ERR_INVALID_ARG, "the scaled base overflows");
  out->pairs = rot_dim / 2;
  out->mscale = static_cast<float>(mscale);
  for (int i = 0; i < SP_ROPE_MAX_PAIRS; ++i) {
    if (i >= out->pairs) {
      out->turns[i] = 0;
      continue;
    }
    double w = std::pow(b, -2.0 * i / dim);
    if (scaling == SP_ROPE_LINEAR) w /= factor;
    if (scaling == SP_ROPE_PARTS) {
      double g = (static_cast<double>(original_len) * w / kTau - low_turns) /
                 (high_turns - low_turns);
      g = g < 0 ? 0 : g > 1 ? 1 : g;
      w *= g + (1 - g) / factor;
    }
    out->turns[i] = static_cast<uint64_t>(std::ldexp(w / kTau, 64) + 0.5);   // w <= 1: below 2^62
  }
  return SP_OK;
}

sp_status_t sp_rope_fwd(const void* const* x, int64_t x_ld, int64_t x_head, int64_t b, int64_t s,
                        int64_t heads, int64_t d, int32_t t, sp_dtype_t dtype,
                        const sp_rope_table_t* table, sp_rope_layout_t layout,
                        const int64_t* positions, int64_t first_position,
                        const int32_t* cu_seqlens, int32_t n_seqs, void* const* y, int64_t y_ld,
                        int64_t y_head, int32_t* dev_status, void* stream) {
  return rope(x, x_ld, x_head, b, s, heads, d, t, dtype, table, layout, positions, first_position,
              cu_seqlens, n_seqs, y, y_ld, y_head, dev_status, stream, 1.f);
}

sp_status_t sp_rope_bwd(const void* const* dy, int64_t dy_ld, int64_t dy_head, int64_t b,
                        int64_t s, int64_t heads, int64_t d, int32_t t, sp_dtype_t dtype,
                        const sp_rope_table_t* table, sp_rope_layout_t layout,
                        const int64_t* positions, int64_t first_position,
                        const int32_t* cu_seqlens, int32_t n_seqs, void* const* dx, int64_t dx_ld,
                        int64_t dx_head, int32_t* dev_status, void* stream) {
  return rope(dy, dy_ld, dy_head, b, s, heads, d, t, dtype, table, layout, positions,
              first_position, cu_seqlens, n_seqs, dx, dx_ld, dx_head, dev_status, stream, -1.f);
}

sp_status_t sp_rope_axes_table(const int32_t* sections, int32_t axes, double base,
                               sp_rope_order_t order, sp_rope_frequencies_t frequencies,
                               const double* factors, double mscale, sp_rope_axes_table_t* out) {
  if (out == nullptr || sections == nullptr)
    return fail(SP_ERR_INVALID_ARG, "%s is NULL", out == nullptr ? "out" : "sections");
  if (axes < 1 || axes > SP_ROPE_MAX_AXES)
    return fail(SP_ERR_INVALID_ARG, "axes = %d outside [1, %d]", axes, SP_ROPE_MAX_AXES);
  int64_t pairs = 0;
  for (int k = 0; k < axes; ++k) {
    if (sections[k] < 1)
      return fail(SP_ERR_INVALID_ARG, "sections[%d] = %d must be >= 1", k, sections[k]);
    pairs += sections[k];
  }
  if (pairs > SP_ROPE_MAX_PAIRS)
    return fail(SP_ERR_INVALID_ARG, "%lld pairs above %d", (long long)pairs, SP_ROPE_MAX_PAIRS);
  if (!(base >= 1.0) || !std::isfinite(base)) return fail(SP_ERR_INVALID_ARG, "base must be >= 1");
  if (order != SP_ROPE_BLOCKS && order != SP_ROPE_CYCLIC)
    return fail(SP_ERR_INVALID_ARG, "unknown order %d", (int)order);
  if (frequencies != SP_ROPE_SHARED && frequencies != SP_ROPE_OWN)
    return fail(SP_ERR_INVALID_ARG, "unknown frequencies %d", (int)frequencies);
  if (!std::isfinite(mscale)) return fail(SP_ERR_INVALID_ARG, "mscale must be finite");
  for (int k = 0; k < axes && factors != nullptr; ++k)
    if (!(factors[k] >= 1.0) || !std::isfinite(factors[k]))
      return fail(SP_ERR_INVALID_ARG, "factors[%d] must be >= 1", k);
  const double kTau = 6.283185307179586476925286766559;
  *out = sp_rope_axes_table_t{};
  out->pairs = static_cast<int32_t>(pairs);
  out->axes = axes;
  out->mscale = static_cast<float>(mscale);
  int32_t given[SP_ROPE_MAX_AXES] = {};
  int32_t k = 0;
  for (int i = 0; i < out->pairs; ++i) {
    // blocks: the first axis with a pair left; cyclic: the next one
    if (order == SP_ROPE_CYCLIC && i > 0) k = (k + 1) % axes;
    while (given[k] == sections[k]) k = (k + 1) % axes;
    const double rate = frequencies == SP_ROPE_SHARED
                            ? static_cast<double>(i) / static_cast<double>(pairs)
                            : static_cast<double>(given[k]) / static_cast<double>(sections[k]);
    double w = std::pow(base, -rate);
    if (factors != nullptr) w /= factors[k];
    out->axis[i] = static_cast<uint8_t>(k);
    out->turns[i] = static_cast<uint64_t>(std::ldexp(w / kTau, 64) + 0.5);   // w <= 1: below 2^62
    ++given[k];
  }
  return SP_OK;
}

sp_status_t sp_rope_axes_fwd(const void* const* x, int64_t x_ld, int64_t x_head, int64_t b,
                             int64_t s, int64_t heads, int64_t d, int32_t t, sp_dtype_t dtype,
                             const sp_rope_axes_table_t* table, sp_rope_layout_t layout,
                             const int64_t* positions, void* const* y, int64_t y_ld,
                             int64_t y_head, void* stream) {
  return rope(x, x_ld, x_head, b, s, heads, d, t, dtype, table, layout, positions, 0, nullptr, 0,
              y, y_ld, y_head, nullptr, stream, 1.f);
}

sp_status_t sp_rope_axes_bwd(const void* const* dy, int64_t dy_ld, int64_t dy_head, int64_t b,
                             int64_t s, int64_t heads, int64_t d, int32_t t, sp_dtype_t dtype,
                             const sp_rope_axes_table_t* table, sp_rope_layout_t layout,
                             const int64_t* positions, void* const* dx, int64_t dx_ld,
                             int64_t dx_head, void* stream) {
  return rope(dy, dy_ld, dy_head, b, s, heads, d, t, dtype, table, layout, positions, 0, nullptr,
              0, dx, dx_ld, dx_head, nullptr, stream, -1.f);
}

sp_status_t sp_gated_scan_fwd(const void* const* gate, int64_t gate_ld, const void* const* value,
                              int64_t value_ld, const float* const* h0, int64_t b, int64_t s,
                              int64_t c, int32_t t, sp_dtype_t dtype, int32_t tied,
                              const int32_t* cu_seqlens, int32_t n_seqs, void* const* y,
                              int64_t y_ld, float* const* hT, float* const* states,
                              int32_t* dev_status, void* stream) {
  sp_status_t st;
  if (take_injected(&st)) return st;
  const ScanCall k{b, s, c, t, dtype, cu_seqlens, n_seqs};
  if ((st = check_scan(k, dev_status)) != SP_OK) return st;
  const int64_t rows = b * s;
  if ((st = check_ld(gate_ld, c, rows, "gate_ld")) != SP_OK) return st;
  if ((st = check_ld(value_ld, c, rows, "value_ld")) != SP_OK) return st;
  if ((st = check_ld(y_ld, c, rows, "y_ld")) != SP_OK) return st;
  if (b == 0) return SP_OK;
  if (h0 != nullptr && (st = check_ranks(h0, t, "h0")) != SP_OK) return st;
  if (hT != nullptr && (st = check_ranks(hT, t, "hT")) != SP_OK) return st;
  if (rows > 0) {
    if ((st = check_ranks(gate, t, "gate")) != SP_OK) return st;
    if ((st = check_ranks(value, t, "value")) != SP_OK) return st;
    if ((st = check_ranks(y, t, "y")) != SP_OK) return st;
    if (states != nullptr && (st = check_ranks(states, t, "states")) != SP_OK) return st;
  }
  const int size = elem_size(dtype);
  const size_t state_bytes = static_cast<size_t>(k.seqs() * c) * 4;
  const size_t runs = static_cast<size_t>((s + kScanRun - 1) / kScanRun);
  Ranges rg;
  for (int r = 0; r < t; ++r) {
    if (rows > 0) {
      rg.add_rows(gate[r], rows, gate_ld * size, c * size, false, "gate", r);
      rg.add_rows(value[r], rows, value_ld * size, c * size, false, "value", r);
      rg.add_rows(y[r], rows, y_ld * size, c * size, true, "y", r);
      if (states != nullptr) rg.add(states[r], b * runs * c * 4, true, "states", r);
    }
    if (h0 != nullptr && !(hT != nullptr && hT[r] == h0[r]))
      rg.add(h0[r], state_bytes, false, "h0", r);
    if (hT != nullptr) rg.add(hT[r], state_bytes, true, "hT", r);
  }
  if (cu_seqlens != nullptr) rg.add(cu_seqlens, (n_seqs + size_t(1)) * 4, false, "cu_seqlens", 0);
  if ((st = rg.check()) != SP_OK) return st;
  if (rows == 0) return pass_states(k, h0, hT, stream);

  ScanParams P{};
  fill_scan(&P, k, gate, gate_ld, value, value_ld, h0, tied, dev_status);
  for (int r = 0; r < t; ++r) {
    P.out[r] = static_cast<char*>(y[r]);
    P.hT[r] = hT != nullptr ? hT[r] : nullptr;
    P.states[r] = states != nullptr ? states[r] : nullptr;
  }
  P.ld_out = static_cast<uint32_t>(y_ld * size);
  const cudaError_t e = launch_scan_fwd(P, dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SP_OK : fail_cuda(e, "sp_gated_scan_fwd launch");
}

sp_status_t sp_gated_scan_bwd(const void* const* gate, int64_t gate_ld, const void* const* value,
                              int64_t value_ld, const float* const* h0,
                              const float* const* states, const void* const* dy, int64_t dy_ld,
                              const float* const* dhT, int64_t b, int64_t s, int64_t c, int32_t t,
                              sp_dtype_t dtype, int32_t tied, const int32_t* cu_seqlens,
                              int32_t n_seqs, void* const* dgate, int64_t dgate_ld,
                              void* const* dvalue, int64_t dvalue_ld, float* const* dh0,
                              int32_t* dev_status, void* stream) {
  sp_status_t st;
  if (take_injected(&st)) return st;
  const ScanCall k{b, s, c, t, dtype, cu_seqlens, n_seqs};
  if ((st = check_scan(k, dev_status)) != SP_OK) return st;
  const int64_t rows = b * s;
  const int64_t lds[] = {gate_ld, value_ld, dy_ld, dgate_ld, dvalue_ld};
  const char* names[] = {"gate_ld", "value_ld", "dy_ld", "dgate_ld", "dvalue_ld"};
  for (int i = 0; i < 5; ++i)
    if ((st = check_ld(lds[i], c, rows, names[i])) != SP_OK) return st;
  if (b == 0) return SP_OK;
  if (h0 != nullptr && (st = check_ranks(h0, t, "h0")) != SP_OK) return st;
  if (dhT != nullptr && (st = check_ranks(dhT, t, "dhT")) != SP_OK) return st;
  if (dh0 != nullptr && (st = check_ranks(dh0, t, "dh0")) != SP_OK) return st;
  if (rows > 0) {
    if ((st = check_ranks(gate, t, "gate")) != SP_OK) return st;
    if ((st = check_ranks(value, t, "value")) != SP_OK) return st;
    if ((st = check_ranks(states, t, "states")) != SP_OK) return st;
    if ((st = check_ranks(dy, t, "dy")) != SP_OK) return st;
    if ((st = check_ranks(dgate, t, "dgate")) != SP_OK) return st;
    if ((st = check_ranks(dvalue, t, "dvalue")) != SP_OK) return st;
  }
  const int size = elem_size(dtype);
  const size_t state_bytes = static_cast<size_t>(k.seqs() * c) * 4;
  const size_t runs = static_cast<size_t>((s + kScanRun - 1) / kScanRun);
  Ranges rg;
  for (int r = 0; r < t; ++r) {
    if (rows > 0) {
      rg.add_rows(gate[r], rows, gate_ld * size, c * size, false, "gate", r);
      rg.add_rows(value[r], rows, value_ld * size, c * size, false, "value", r);
      rg.add_rows(dy[r], rows, dy_ld * size, c * size, false, "dy", r);
      rg.add(states[r], b * runs * c * 4, false, "states", r);
      rg.add_rows(dgate[r], rows, dgate_ld * size, c * size, true, "dgate", r);
      rg.add_rows(dvalue[r], rows, dvalue_ld * size, c * size, true, "dvalue", r);
    }
    if (h0 != nullptr) rg.add(h0[r], state_bytes, false, "h0", r);
    if (dhT != nullptr) rg.add(dhT[r], state_bytes, false, "dhT", r);
    if (dh0 != nullptr) rg.add(dh0[r], state_bytes, true, "dh0", r);
  }
  if (cu_seqlens != nullptr) rg.add(cu_seqlens, (n_seqs + size_t(1)) * 4, false, "cu_seqlens", 0);
  if ((st = rg.check()) != SP_OK) return st;
  if (rows == 0) return pass_states(k, dhT, dh0, stream);

  ScanParams P{};
  fill_scan(&P, k, gate, gate_ld, value, value_ld, h0, tied, dev_status);
  for (int r = 0; r < t; ++r) {
    P.dy[r] = static_cast<const char*>(dy[r]);
    P.out[r] = static_cast<char*>(dgate[r]);
    P.dvalue[r] = static_cast<char*>(dvalue[r]);
    P.dhT[r] = dhT != nullptr ? dhT[r] : nullptr;
    P.hT[r] = dh0 != nullptr ? dh0[r] : nullptr;
    P.states[r] = const_cast<float*>(states[r]);
  }
  P.ld_dy = static_cast<uint32_t>(dy_ld * size);
  P.ld_out = static_cast<uint32_t>(dgate_ld * size);
  P.ld_dvalue = static_cast<uint32_t>(dvalue_ld * size);
  const cudaError_t e = launch_scan_bwd(P, dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SP_OK : fail_cuda(e, "sp_gated_scan_bwd launch");
}

sp_status_t sp_group_norm_fwd(const void* const* x, int64_t x_ld, const void* gamma,
                              const void* beta, int64_t n, int64_t l, int64_t c, int64_t groups,
                              int32_t t, sp_dtype_t dtype, float eps, sp_norm_t norm, sp_act_t act,
                              void* const* y, int64_t y_ld, float* const* mean,
                              float* const* rstd, void* stream) {
  sp_status_t st;
  if (take_injected(&st)) return st;
  if ((st = check_group(n, l, c, groups, t, dtype)) != SP_OK) return st;
  if ((st = check_act(norm, act)) != SP_OK) return st;
  if (!(eps > 0.f) || !std::isfinite(eps)) return fail(SP_ERR_INVALID_ARG, "eps must be > 0");
  const int64_t rows = n * l;
  if ((st = check_ld(x_ld, c, rows, "x_ld")) != SP_OK) return st;
  if ((st = check_ld(y_ld, c, rows, "y_ld")) != SP_OK) return st;
  if (rows == 0) return SP_OK;
  const bool ln = norm == SP_NORM_LAYERNORM;
  if ((st = check_ranks(x, t, "x")) != SP_OK) return st;
  if ((st = check_ranks(y, t, "y")) != SP_OK) return st;
  if ((st = check_stats(rstd, t, "rstd")) != SP_OK) return st;
  if (ln && (st = check_stats(mean, t, "mean")) != SP_OK) return st;
  if ((st = check_param(gamma, "gamma")) != SP_OK) return st;
  if (ln && (st = check_param(beta, "beta")) != SP_OK) return st;
  const int size = elem_size(dtype);
  Ranges rg;
  for (int r = 0; r < t; ++r) {
    rg.add_rows(x[r], rows, x_ld * size, c * size, false, "x", r);
    rg.add_rows(y[r], rows, y_ld * size, c * size, true, "y", r);
    rg.add(rstd[r], n * groups * 4, true, "rstd", r);
    if (ln) rg.add(mean[r], n * groups * 4, true, "mean", r);
  }
  rg.add(gamma, t * c * size, false, "gamma", 0);
  if (ln) rg.add(beta, t * c * size, false, "beta", 0);
  if ((st = rg.check()) != SP_OK) return st;

  GroupNormParams P{};
  fill_group(&P, n, l, c, groups, t, norm, act, gamma, ln ? beta : nullptr);
  for (int r = 0; r < t; ++r) {
    P.x[r] = static_cast<const char*>(x[r]);
    P.out[r] = static_cast<char*>(y[r]);
    P.mean[r] = ln ? mean[r] : nullptr;
    P.rstd[r] = rstd[r];
  }
  P.ld_x = x_ld * size;
  P.ld_out = y_ld * size;
  P.eps = eps;
  const cudaError_t e = launch_group_norm_fwd(P, dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SP_OK : fail_cuda(e, "sp_group_norm_fwd launch");
}

size_t sp_group_norm_bwd_workspace_bytes(int64_t n, int64_t l, int64_t c, int64_t groups,
                                         int32_t t, sp_dtype_t dtype) {
  if (check_group(n, l, c, groups, t, dtype) != SP_OK || n * l == 0) return 0;
  const GroupShape s = group_norm_shape(n, l, static_cast<int>(c), static_cast<int>(groups), t,
                                        dtype, true);
  return static_cast<size_t>(s.parts) * 2 * static_cast<size_t>(t * c) * sizeof(float);
}

sp_status_t sp_debug_group_norm_shape(int64_t n, int64_t l, int64_t c, int64_t groups, int32_t t,
                                      sp_dtype_t dtype, int32_t backward, int64_t* out) {
  sp_status_t st;
  if ((st = check_group(n, l, c, groups, t, dtype)) != SP_OK) return st;
  if (n * l == 0 || out == nullptr)
    return fail(SP_ERR_INVALID_ARG, "sp_debug_group_norm_shape: bad arguments");
  const GroupShape s = group_norm_shape(n, l, static_cast<int>(c), static_cast<int>(groups), t,
                                        dtype, backward != 0);
  const int64_t v[8] = {s.form, s.threads, s.cluster, s.cols,
                        s.slabs, s.rows, s.parts, static_cast<int64_t>(s.smem)};
  for (int i = 0; i < 8; ++i) out[i] = v[i];
  return SP_OK;
}

sp_status_t sp_group_norm_bwd(const void* const* dy, int64_t dy_ld, const void* const* x,
                              int64_t x_ld, const float* const* mean, const float* const* rstd,
                              const void* gamma, const void* beta, int64_t n, int64_t l, int64_t c,
                              int64_t groups, int32_t t, sp_dtype_t dtype, sp_norm_t norm,
                              sp_act_t act, void* const* dx, int64_t dx_ld, float* dgamma,
                              float* dbeta, void* workspace, size_t workspace_bytes,
                              void* stream) {
  sp_status_t st;
  if (take_injected(&st)) return st;
  if ((st = check_group(n, l, c, groups, t, dtype)) != SP_OK) return st;
  if ((st = check_act(norm, act)) != SP_OK) return st;
  const int64_t rows = n * l;
  if ((st = check_ld(dy_ld, c, rows, "dy_ld")) != SP_OK) return st;
  if ((st = check_ld(x_ld, c, rows, "x_ld")) != SP_OK) return st;
  if ((st = check_ld(dx_ld, c, rows, "dx_ld")) != SP_OK) return st;
  const bool ln = norm == SP_NORM_LAYERNORM;
  if (!ln) dbeta = nullptr;
  if (dgamma != nullptr && !aligned16(dgamma)) return fail(SP_ERR_MISALIGNED, "dgamma misaligned");
  if (dbeta != nullptr && !aligned16(dbeta)) return fail(SP_ERR_MISALIGNED, "dbeta misaligned");
  const size_t width = static_cast<size_t>(t * c) * sizeof(float);
  if (rows == 0) {
    // no row: the parameter gradients are exact zeros, nothing else is touched
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (dgamma != nullptr) e = cudaMemsetAsync(dgamma, 0, width, cs);
    if (e == cudaSuccess && dbeta != nullptr) e = cudaMemsetAsync(dbeta, 0, width, cs);
    return e == cudaSuccess ? SP_OK : fail_cuda(e, "sp_group_norm_bwd zero fill");
  }
  if ((st = check_ranks(dy, t, "dy")) != SP_OK) return st;
  if ((st = check_ranks(x, t, "x")) != SP_OK) return st;
  if ((st = check_ranks(dx, t, "dx")) != SP_OK) return st;
  if ((st = check_stats(const_cast<float* const*>(rstd), t, "rstd")) != SP_OK) return st;
  if (ln && (st = check_stats(const_cast<float* const*>(mean), t, "mean")) != SP_OK) return st;
  if ((st = check_param(gamma, "gamma")) != SP_OK) return st;
  if (ln && (st = check_param(beta, "beta")) != SP_OK) return st;
  size_t need = 0;
  if (dgamma != nullptr || dbeta != nullptr) {
    need = sp_group_norm_bwd_workspace_bytes(n, l, c, groups, t, dtype);
    if (workspace == nullptr || workspace_bytes < need)
      return fail(SP_ERR_INVALID_ARG, "workspace of %zu bytes needed (got %zu)", need,
                  workspace == nullptr ? (size_t)0 : workspace_bytes);
    if (!aligned16(workspace)) return fail(SP_ERR_MISALIGNED, "workspace misaligned");
  }
  const int size = elem_size(dtype);
  Ranges rg;
  for (int r = 0; r < t; ++r) {
    rg.add_rows(dy[r], rows, dy_ld * size, c * size, false, "dy", r);
    rg.add_rows(x[r], rows, x_ld * size, c * size, false, "x", r);
    rg.add(rstd[r], n * groups * 4, false, "rstd", r);
    if (ln) rg.add(mean[r], n * groups * 4, false, "mean", r);
    rg.add_rows(dx[r], rows, dx_ld * size, c * size, true, "dx", r);
  }
  rg.add(gamma, t * c * size, false, "gamma", 0);
  if (ln) rg.add(beta, t * c * size, false, "beta", 0);
  rg.add(dgamma, width, true, "dgamma", 0);
  rg.add(dbeta, width, true, "dbeta", 0);
  if (need > 0) rg.add(workspace, need, true, "workspace", 0);
  if ((st = rg.check()) != SP_OK) return st;

  GroupNormParams P{};
  fill_group(&P, n, l, c, groups, t, norm, act, gamma, ln ? beta : nullptr);
  for (int r = 0; r < t; ++r) {
    P.x[r] = static_cast<const char*>(x[r]);
    P.dy[r] = static_cast<const char*>(dy[r]);
    P.out[r] = static_cast<char*>(dx[r]);
    P.mean[r] = ln ? const_cast<float*>(mean[r]) : nullptr;
    P.rstd[r] = const_cast<float*>(rstd[r]);
  }
  P.ld_x = x_ld * size;
  P.ld_dy = dy_ld * size;
  P.ld_out = dx_ld * size;
  P.ws = static_cast<float*>(workspace);
  const cudaError_t e =
      launch_group_norm_bwd(P, dtype, dgamma, dbeta, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SP_OK : fail_cuda(e, "sp_group_norm_bwd launch");
}

}  // extern "C"
