// Products of MXFP4 operands on the scaled matrix instruction (gfx950), shared by the kernels
// of the 4-bit head.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes 32 e2m1 codes of a row and their block's scale byte
// per lane (lane l: row l % 32, one block of the two that a call covers) and accumulates in
// fp32: products of codes are exact, and nothing is rounded before the output.  The
// contraction's order is free as long as both operands agree, so the blocks are dealt out to
// suit the loads: of the 8 blocks in 256 K (128 bytes of codes, one step), the lower half-wave
// takes blocks 0-3 and the upper 4-7, one each per instruction.  A lane's four scale bytes of a
// step are then one aligned dword, and the instruction picks byte kk.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "ops_internal.h"
#include "tile_device.h"

namespace flce {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kE2m1 = 4;  // the instruction's format code of e2m1

// D += A B^T of 32 rows each over 64 K, with scale byte kk of sa and sb.
template <int kk>
__device__ __forceinline__ f32x16 mx_mfma(u32x4 a, u32x4 b, f32x16 c, int sa, int sb) {
  const i32x8 a8 = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 b8 = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, kE2m1, kE2m1, kk, sa, kk, sb);
}

// Chunk c (16 bytes, one block) of row r of a code tile in LDS sits at position c ^ mx_swz(r)
// of the row's 128 bytes: the 16 rows that one cycle of a fragment read serves land on 16
// distinct 16-byte bank groups, and the swizzle is the same for rows 32 apart, so a fragment's
// 32-row block is an immediate offset.
__device__ __forceinline__ int mx_swz(int r) { return (r ^ ((r >> 3) & 3)) & 7; }

// Offset of a row's scale bytes.
__device__ __forceinline__ long mx_scale_row(const MxScaleLayout& l, long row) {
  return (row >> 8) * l.tile_stride + (row & 255) * l.row_stride;
}

}  // namespace flce
