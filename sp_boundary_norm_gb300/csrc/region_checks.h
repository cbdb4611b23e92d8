// Checks of arguments that the entry points between g and the next g* share.
#pragma once

#include "host_common.h"

namespace spb {

constexpr int64_t kMostElements = int64_t(1) << 48;   // of one rank's tensor, strides included

inline int elem_size(sp_dtype_t dtype) { return dtype == SP_F32 ? 4 : 2; }

inline sp_status_t check_common(int32_t t, sp_dtype_t dtype, const int32_t* dev_status) {
  if (t < 1 || t > SP_MAX_RANKS)
    return fail(SP_ERR_INVALID_ARG, "t = %d outside [1, %d]", t, SP_MAX_RANKS);
  if (dtype != SP_BF16 && dtype != SP_F16 && dtype != SP_F32)
    return fail(SP_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
  if (dev_status != nullptr && (reinterpret_cast<uintptr_t>(dev_status) & 3u))
    return fail(SP_ERR_MISALIGNED, "dev_status misaligned");
  return SP_OK;
}

inline sp_status_t check_seqs(int64_t b, int64_t s, const int32_t* cu_seqlens, int32_t n_seqs) {
  if (b < 0 || s < 0) return fail(SP_ERR_INVALID_ARG, "negative b or s");
  if (b > kMostElements || s > kMostElements || (s > 0 && b > kMostElements / s))
    return fail(SP_ERR_INVALID_ARG, "b*s overflows");
  if (cu_seqlens == nullptr) return SP_OK;
  if (b != 1)
    return fail(SP_ERR_INVALID_ARG, "cu_seqlens requires b == 1 (got %lld)", (long long)b);
  if (n_seqs < 1) return fail(SP_ERR_INVALID_ARG, "n_seqs = %d must be >= 1", n_seqs);
  if (s > 0x7FFFFFFF)
    return fail(SP_ERR_INVALID_ARG, "cu_seqlens counts to 2^31 - 1 tokens (got %lld)", (long long)s);
  if (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)
    return fail(SP_ERR_MISALIGNED, "cu_seqlens not 4-byte aligned");
  return SP_OK;
}

template <typename T>
inline sp_status_t check_ranks(T* const* arr, int t, const char* what) {
  if (arr == nullptr) return fail(SP_ERR_INVALID_ARG, "%s array is NULL", what);
  for (int i = 0; i < t; ++i) {
    if (arr[i] == nullptr) return fail(SP_ERR_INVALID_ARG, "%s[%d] is NULL", what, i);
    if (!aligned16(arr[i])) return fail(SP_ERR_MISALIGNED, "%s[%d] misaligned", what, i);
  }
  return SP_OK;
}

constexpr int64_t kMostLd = int64_t(1) << 28;   // a row stride in bytes fits 32 bits

// A row stride: a multiple of 8 elements, at least the row, no overflow.
inline sp_status_t check_ld(int64_t ld, int64_t width, int64_t rows, const char* what) {
  if (ld < width || ld % 8 != 0)
    return fail(SP_ERR_INVALID_ARG, "%s = %lld must be a multiple of 8 and at least %lld", what,
                (long long)ld, (long long)width);
  if (rows > 0 && ld > kMostElements / rows)
    return fail(SP_ERR_INVALID_ARG, "%s: the tensor's extent overflows", what);
  if (ld > kMostLd)
    return fail(SP_ERR_UNSUPPORTED, "%s = %lld above %lld", what, (long long)ld,
                (long long)kMostLd);
  return SP_OK;
}

}  // namespace spb
