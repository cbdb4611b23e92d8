// Parameters and launchers of the operators between g and the next g*.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sp_boundary.h"
#include "sp_internal.h"

namespace spb {

// ------------------------------------------------------------------ rotary --
struct RopeParams {
  const char* x[SP_MAX_RANKS];
  char* y[SP_MAX_RANKS];
  int64_t x_row, x_head, y_row, y_head;   // bytes between rows (tokens) and heads
  int64_t s, tokens;                      // tokens of a batch row, of the call
  int32_t all_heads, heads;               // over all ranks, of one rank
  uint32_t heads_magic;                   // ceil(2^32 / heads)
  int32_t half;                           // rotated pairs of a head
  int32_t rest, rest_at, rest_bytes;      // bytes after them to copy (0 in place), the first,
                                          // bytes of one access
  int32_t chunks, chunk_heads;            // pieces of a token's heads, one warp each
  int32_t layout;
  const int64_t* positions;
  int64_t first;
  const int32_t* cu_seqlens;
  int32_t n_seqs;
  float cos_scale, sin_scale;
  int32_t* status;
  uint64_t turns[SP_ROPE_MAX_PAIRS];      // turns per position, fractions of 2^64
};

cudaError_t launch_rope(RopeParams p, int dtype, int vec, cudaStream_t st);

// ---------------------------------------------------------- gated recurrence --
constexpr int kScanRun = 16;        // tokens of one thread, and of one saved state
constexpr int kScanChannels = 64;   // channels of a block: two a lane
constexpr int kScanWarps = 4;       // of a small block, at most
constexpr int kScanWideWarps = 12;  // of a block that has an SM to itself
constexpr size_t kScanMaxShared = 232448;   // bytes that a block may ask for
constexpr int kScanMaxCluster = 16;

struct ScanParams {
  const char* gate[SP_MAX_RANKS];
  const char* value[SP_MAX_RANKS];
  const char* dy[SP_MAX_RANKS];
  char* out[SP_MAX_RANKS];            // forward: y; backward: dgate
  char* dvalue[SP_MAX_RANKS];
  const float* h0[SP_MAX_RANKS];      // NULL: zero
  const float* dhT[SP_MAX_RANKS];     // NULL: zero
  float* hT[SP_MAX_RANKS];            // forward: hT; backward: dh0; NULL: not wanted
  float* states[SP_MAX_RANKS];        // NULL (forward): not wanted
  uint32_t ld_gate, ld_value, ld_dy, ld_out, ld_dvalue;   // bytes between tokens
  int64_t s;
  int32_t b, c, t, slabs;
  int32_t tied, cluster;
  const int32_t* cu_seqlens;
  int32_t n_seqs;
  int32_t* status;
  int32_t withhold;                   // test hook: block 0 does not send this step's map; -1
};

cudaError_t launch_scan_fwd(ScanParams p, int dtype, cudaStream_t st);
cudaError_t launch_scan_bwd(ScanParams p, int dtype, cudaStream_t st);
// -------------------------------------------------------------- group norm --
constexpr int kGroupThreads = 512;      // most threads of a block: cols <= this
constexpr int kGroupMaxCluster = 16;

struct GroupNormParams {
  const char* x[SP_MAX_RANKS];
  const char* dy[SP_MAX_RANKS];
  char* out[SP_MAX_RANKS];              // forward: y; backward: dx
  float* mean[SP_MAX_RANKS];            // LayerNorm: written forward, read backward
  float* rstd[SP_MAX_RANKS];
  const char* gamma;                    // [t * c]
  const char* beta;                     // [t * c], LayerNorm
  int64_t ld_x, ld_dy, ld_out;          // bytes between rows
  int64_t n, l;                         // samples, rows of a sample
  int32_t c, t, groups, norm, act;
  float eps, count, count_inv;          // l * channels of a group, 1 / that
  // the split of a call, chosen on the host
  int32_t q;                            // 8-channel vectors of a group
  int32_t cols, slabs;                  // vectors of a slab (whole groups), slabs of a row
  int32_t rows;                         // rows (rows form: teams) side by side in a block
  int32_t samples;                      // tiles: samples of a tile
  int32_t lanes;                        // tiles: lanes that sum one group of one sample
  int64_t parts;                        // blocks of one rank's slab (units: of all its samples)
  int32_t cluster;                      // units: blocks of a sample
  float* ws;                            // backward: [parts][2][t * c]
  int32_t has_params;                   // backward: dgamma / dbeta wanted
};

// The split of a call (see GroupNormParams).
constexpr int kRowForm = 0, kTileForm = 1, kHeldForm = 2, kUnitForm = 3;
struct GroupShape {
  int form, mode;
  int cols, slabs, rows, threads, samples, lanes, cluster;
  int64_t parts;
  size_t smem;
  bool roomy;                           // units: an SM holds two blocks at most
};

GroupShape group_norm_shape(int64_t n, int64_t l, int c, int groups, int t, int dtype, bool bwd);
// Launches a form's kernel, filling p's split.
cudaError_t launch_group(const void* fn, GroupNormParams* p, const GroupShape& s, cudaStream_t st);
cudaError_t launch_group_norm_fwd(GroupNormParams p, int dtype, cudaStream_t st);
cudaError_t launch_group_norm_bwd(GroupNormParams p, int dtype, float* dgamma, float* dbeta,
                                  cudaStream_t st);

}  // namespace spb
