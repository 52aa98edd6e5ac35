// Internal interface between the libflce host code and the kernels of the operators
// around the head: layer norm, microscaled formats, the head with 4-bit weights.
// Not installed; not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "flce_internal.h"
#include "mx_layout.h"

namespace flce {

struct NormFwdArgs {
  const void* x;
  long ldx;                // elements between rows
  const void* weight;      // [H] or nullptr (1)
  const void* bias;        // [H] or nullptr (0)
  int param_dtype;
  long M;
  int H;
  float eps;
  void* y;
  long ldy;
  float* mean;
  float* rstd;
  int fmt;                 // checkpoint format, kMxNone for none
  uint8_t* codes;
  uint8_t* scales;
};

struct NormBwdArgs {
  const void* dy;
  long lddy;
  const void* x;           // the input, or nullptr: codes and scales of it
  long ldx;
  int fmt;
  const uint8_t* codes;
  const uint8_t* scales;
  const void* weight;      // [H] or nullptr (1)
  int param_dtype;
  const float* mean;
  const float* rstd;
  long M;
  int H;
  void* dx;
  long lddx;
  bool params;             // whether the partial sums are wanted
  float* part;             // [2][groups][H] partial sums of dweight and dbias
  int groups;              // workgroups of the row kernel = rows of each partial array
};

struct NormReduceArgs {
  const float* part;
  int groups;
  int H;
  void* dweight;           // [H] or nullptr
  void* dbias;
  int param_dtype;
};

// Workgroups of the backward's row kernel for a shape (they share the rows between them and
// leave one partial sum each).
int norm_bwd_groups(long M, int H);
hipError_t launch_norm_fwd(const NormFwdArgs& a, int x_dtype, int y_dtype, bool vec, hipStream_t s);
hipError_t launch_norm_bwd(const NormBwdArgs& a, int x_dtype, int dy_dtype, int dx_dtype, bool vec,
                           hipStream_t s);
hipError_t launch_norm_reduce(const NormReduceArgs& a, hipStream_t s);

// Where the scale bytes of a microscaled matrix lie: those of blocks 16 q .. 16 q + 15 of row
// r are the 16 bytes at (r / 256) tile_stride + (r % 256) row_stride + q quad_stride.  The
// public form is row-major; the tile kernels read a form in which the rows of a 256-row tile
// are side by side and a tile's bytes contiguous.
struct MxScaleLayout {
  long row_stride, quad_stride, tile_stride;
};
inline MxScaleLayout mx_row_major(int64_t cols) {
  return {long(mx_scale_bytes(cols)), 16, long(256 * mx_scale_bytes(cols))};
}
inline MxScaleLayout mx_tiled(int64_t cols) { return {16, 16 * 256, long(256 * mx_scale_bytes(cols))}; }

// Scales of `rows` rows to be written in the tile kernels' form (whole 256-row tiles) by
// `groups` workgroups of their own.
struct MxTurn {
  const uint8_t* src;      // row-major
  uint8_t* dst;
  long rows;
  int quads;               // 16-byte pieces of a row
  unsigned groups;         // 0: nothing to do
};
inline MxTurn mx_turn(const uint8_t* src, uint8_t* dst, int64_t rows, int64_t cols) {
  const int64_t quads = mx_scale_bytes(cols) / 16, need = ((rows + 7) / 8 * ((quads + 7) / 8) + 3) / 4;
  return {src, dst, long(rows), int(quads), unsigned(need < 4096 ? need : 4096)};
}

struct MxQuantArgs {
  const void* x;           // quantise: the matrix; dequantise: unused
  long ldx;
  void* out;               // dequantise: the values
  long ldo;
  uint8_t* codes;
  uint8_t* scales;
  long rows;
  long cols;
  MxScaleLayout layout;
  unsigned long long* clear;  // quantise: 8 counters to zero for a later launch, or nullptr
  MxTurn turn;             // quantise: another matrix's scales on the way
};
hipError_t launch_mx_quantize(const MxQuantArgs& a, int dtype, int fmt, bool vec, hipStream_t s);
hipError_t launch_mx_dequantize(const MxQuantArgs& a, int dtype, int fmt, bool vec, hipStream_t s);

// The head with 4-bit weights: X and W as MXFP4 codes and scales.  Calls of at most
// kMxStreamTokens tokens always run the kernels that stream W past the tokens, of which
// kMxStreamResident workgroups run at once (those of 128 vocabulary rows).
constexpr int64_t kMxStreamTokens = 128, kMxStreamResident = 512;
struct MxOperand {
  const uint8_t* codes;
  const uint8_t* scales;
  MxScaleLayout layout;
};
// A decoding step's tokens are quantised by the product's workgroups themselves where their
// codes (rows padded to 1024 K) take at most kMxOwnBytes.
constexpr int kMxOwnBytes = 8192;
constexpr bool mx_stream_owns(int64_t M, int64_t H) {
  return M <= 8 && M * ((mx_blocks(H) + 31) / 32 * 512) <= kMxOwnBytes;
}
struct MxLogitsArgs {
  const uint16_t* X;       // bf16 [M, H], if mx_stream_owns (x is then unused); else nullptr
  MxOperand x, w;
  int M, H, V;
  float scale;
  void* out;               // [M, V] logits
  long ldo;
  int out_dtype;
  long call_M;             // rows of the whole call, of which M are this launch
  int n_mt, n_vt;          // 256 x 256 tiles (the tile kernel)
};

// Log-prob partials: entry (vocabulary tile j, token m) of each array at j * tile_stride +
// m * token_stride.
struct MxFwdArgs {
  const uint16_t* X;       // as in MxLogitsArgs
  MxOperand x, w;
  const int64_t* targets;
  int M, H, V;
  int64_t ignore_index;
  float scale;
  int n_mt, n_vt;          // n_vt: vocabulary tiles that leave partials
  long tile_stride, token_stride;
  long call_M;             // rows of the whole call, of which M are this wave
  float* part_m;
  float* part_s;
  float* part_u;           // nullptr without entropy
  float* logprob;
  float* lse;
  float* entropy;
};

// The kernels for few tokens: vocabulary rows a workgroup takes, for a call of M tokens.
int mx_stream_rows(long M, int V);
hipError_t launch_mx_stream_logits(const MxLogitsArgs& a, hipStream_t s);
hipError_t launch_mx_stream_fwd(const MxFwdArgs& a, hipStream_t s);
hipError_t launch_mx_tile_logits(const MxLogitsArgs& a, hipStream_t s);
hipError_t launch_mx_tile_fwd(const MxFwdArgs& a, TileQueue tq, hipStream_t s);
// Target logits and the merge of the partials into logprob, lse and entropy.
hipError_t launch_mx_merge(const MxFwdArgs& a, hipStream_t s);

}  // namespace flce
