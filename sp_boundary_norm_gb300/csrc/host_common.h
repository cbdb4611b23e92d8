// Helpers shared by the host sides of the entry points (defined in api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sp_boundary.h"

namespace spb {

// Sets the thread's sp_last_error() text; returns `code`.
sp_status_t fail(sp_status_t code, const char* fmt, ...);
sp_status_t fail_cuda(cudaError_t e, const char* where);
// An armed sp_debug_inject: true, and its status in *out.
bool take_injected(sp_status_t* out);
// The step of an armed sp_debug_scan_withhold, or -1.
int32_t take_withheld_step();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A list of device byte ranges; outputs must not overlap anything else.
struct Ranges {
  struct R {
    uintptr_t lo, hi;
    bool out;
    const char* what;
    int idx;
    uintptr_t pitch, width;   // rows of `width` bytes every `pitch` bytes (0: one piece)
  };
  static constexpr int kMost = 256;   // 16 ranks' tensors of any entry point
  R v[kMost];
  int n = 0;
  void put(const R& r) {
    if (n < kMost) v[n] = r;
    ++n;
  }
  void add(const void* p, size_t bytes, bool out, const char* what, int idx) {
    if (p == nullptr || bytes == 0) return;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    put({lo, lo + bytes, out, what, idx, 0, 0});
  }
  void add_rows(const void* p, size_t rows, size_t pitch, size_t width, bool out, const char* what,
                int idx) {
    if (p == nullptr || rows == 0 || width == 0) return;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    put({lo, lo + (rows - 1) * pitch + width, out, what, idx, pitch, width});
  }
  // Slices of one wider buffer: rows of the same pitch that lie beside each other.
  static bool beside(const R& a, const R& b) {
    if (a.pitch == 0 || a.pitch != b.pitch) return false;
    const uintptr_t off = a.lo <= b.lo ? (b.lo - a.lo) % a.pitch
                                       : (a.pitch - (a.lo - b.lo) % a.pitch) % a.pitch;
    return off >= a.width && off + b.width <= a.pitch;
  }
  sp_status_t check() const {
    if (n > kMost) return fail(SP_ERR_UNSUPPORTED, "more than %d buffers", kMost);
    for (int i = 0; i < n; ++i) {
      if (!v[i].out) continue;
      for (int j = 0; j < n; ++j) {
        if (i == j) continue;
        if (v[i].lo < v[j].hi && v[j].lo < v[i].hi && !beside(v[i], v[j]))
          return fail(SP_ERR_OVERLAP, "output %s[%d] overlaps %s[%d]", v[i].what, v[i].idx,
                      v[j].what, v[j].idx);
      }
    }
    return SP_OK;
  }
};

// Raises a kernel's dynamic shared-memory limit on the current device to `smem`.
cudaError_t ensure_smem_attr(const void* fn, size_t smem);

// Prepares kernel `fn` for clusters of `cluster` blocks of that size on the
// current device; *fit: how many the GPU holds at once.  Remembered.
cudaError_t max_clusters(const void* fn, int threads, size_t smem, int cluster, int* fit);

}  // namespace spb
