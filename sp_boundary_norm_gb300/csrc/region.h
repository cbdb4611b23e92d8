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

// Several axes: `positions` is [axes][tokens], and every pair follows one axis.
struct RopeAxesParams : RopeParams {
  uint8_t axis[SP_ROPE_MAX_PAIRS];
};

cudaError_t launch_rope(const RopeParams& p, int dtype, int vec, cudaStream_t st);
cudaError_t launch_rope_axes(const RopeAxesParams& p, int dtype, int vec, cudaStream_t st);

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


// ------------------------------------------------------- causal convolution --
struct ConvParams {
  const char* x[SP_MAX_RANKS];
  const char* dy[SP_MAX_RANKS];
  char* out[SP_MAX_RANKS];              // forward: y; backward: dx
  const char* x0[SP_MAX_RANKS];         // NULL: zero
  const char* dxT[SP_MAX_RANKS];        // NULL: zero
  char* xT[SP_MAX_RANKS];               // forward: xT; backward: dx0; NULL: not wanted
  const char* weight;                   // [t * c][width]
  const char* bias;                     // [t * c] or NULL
  int64_t ld_x, ld_dy, ld_out;          // bytes between tokens
  int64_t s;                            // tokens of a batch row
  int32_t b, c, t, width, act;
  const int32_t* cu_seqlens;
  int32_t n_seqs;
  int32_t* status;
  // the split of a call
  int32_t vecs, lanes;                  // vectors of a token; threads side by side on them
  int32_t slabs;                        // pieces of `lanes` vectors of a token
  int32_t run;                          // tokens of a thread's run
  int64_t runs;                         // of a batch row
  int32_t parts;                        // backward: blocks of one slab, [parts][t * c][width + 1]
  float* ws;                            // NULL: no parameter gradient wanted
};

cudaError_t launch_conv_fwd(ConvParams p, int dtype, cudaStream_t st);
cudaError_t launch_conv_bwd(ConvParams p, int dtype, float* dweight, float* dbias,
                            cudaStream_t st);
// Blocks of one slab in the backward of a call, which its workspace goes by.
int conv_bwd_parts(int64_t b, int64_t s, int c, int t, int dtype);

// ---------------------------------------------------------- selective scan --
constexpr int kSsmRun = 16;             // tokens of one saved state
constexpr int kSsmTile = 16;            // tokens of a step of a block
constexpr int kSsmStepTokens = 16;      // most tokens of a sequence in a decoding step

struct SsmParams {
  const char* u[SP_MAX_RANKS];
  const char* dt[SP_MAX_RANKS];
  const char* B[SP_MAX_RANKS];
  const char* C[SP_MAX_RANKS];
  const char* z[SP_MAX_RANKS];          // NULL: no gate
  const char* dy[SP_MAX_RANKS];
  char* y[SP_MAX_RANKS];                // forward
  char* du[SP_MAX_RANKS];
  char* ddt[SP_MAX_RANKS];
  char* dB[SP_MAX_RANKS];
  char* dC[SP_MAX_RANKS];
  char* dz[SP_MAX_RANKS];
  float* states[SP_MAX_RANKS];          // forward: NULL if not wanted
  const float* h0[SP_MAX_RANKS];        // NULL: zero
  const float* dhT[SP_MAX_RANKS];       // NULL: zero
  float* hT[SP_MAX_RANKS];              // forward: hT; backward: dh0; NULL: not wanted
  const float* A;                       // [t * c][n]
  const float* D;                       // [t * c] or NULL
  const float* dt_bias;                 // [t * c] or NULL
  int64_t ld_u, ld_dt, ld_B, ld_C, ld_z, ld_dy, ld_y;     // bytes between tokens
  int64_t ld_du, ld_ddt, ld_dB, ld_dC, ld_dz;
  int64_t s;
  int32_t b, c, t, n, groups, softplus, gated;
  const int32_t* cu_seqlens;
  int32_t n_seqs;
  int32_t* status;
  // the split of a call
  int32_t slabs;                        // blocks of a group's channels
  int32_t chunks;                       // pieces of a batch row that run side by side
  int64_t chunk_len;                    // their tokens, a multiple of kSsmTile
  float* carry;                         // [b][chunks][t * c][n]: the state (backward: its
                                        // gradient) that enters a chunk
  float* steps;                         // [b][chunks][t * c]: the sum of a chunk's steps
  float* partial_bc;                    // backward: [t * groups * slabs][b * s][2n], or NULL
  float* partial_params;                // backward: [b * chunks][t * c][n + 2], or NULL
};

// How a call is split on the current device.
struct SsmSplit {
  int32_t slabs, chunks;
  int64_t chunk_len;
  size_t carry, steps, partial_bc, partial_params;   // floats of each
  size_t bytes() const { return (carry + steps + partial_bc + partial_params) * 4; }
};
SsmSplit ssm_split(int64_t b, int64_t s, int64_t c, int n, int groups, int t, bool bwd);

cudaError_t launch_ssm_fwd(const SsmParams& p, int dtype, cudaStream_t st);
cudaError_t launch_ssm_step(const SsmParams& p, int dtype, cudaStream_t st);
struct SsmParamGrads {
  float* dA;
  float* dD;
  float* ddt_bias;
};
cudaError_t launch_ssm_bwd(const SsmParams& p, int dtype, const SsmParamGrads& g, cudaStream_t st);

}  // namespace spb
