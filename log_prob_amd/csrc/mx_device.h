// Microscaled formats on the device (gfx950): blocks of 32 consecutive elements of a row
// share one power-of-two scale 2^(byte - 127); the scale is the smallest one at which no
// element of the block exceeds the element format's largest value, so nothing saturates,
// and elements are rounded to nearest, ties to even.  A thread holds 8 consecutive elements
// (a quarter block), and the four threads of a block are the four lanes of a quad.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_internal.h"

namespace flce {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Two floats as a bf16 pair, rounded to nearest even (a in the low half).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Element types of matrices in memory.
struct Bf16 {
  typedef uint16_t mem;
  static __device__ __forceinline__ float to_f32(uint16_t u) { return __uint_as_float((uint32_t)u << 16); }
  static __device__ __forceinline__ uint16_t from_f32(float f) { return (uint16_t)pack_bf16(f, 0.f); }
};
struct F32 {
  typedef float mem;
  static __device__ __forceinline__ float to_f32(float f) { return f; }
  static __device__ __forceinline__ float from_f32(float f) { return f; }
};

// 16 bytes at the alignment of an element: one access all the same (the device allows
// unaligned ones; element by element, rows of an odd length took 3.5 times as long).
typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));
typedef f32x4_t f32x4_a4 __attribute__((aligned(4)));

// Elements [col, col + 8) of a row of `cols` elements, as they come from memory (so that loads
// can be in flight at few registers' cost) and as floats; elements past the row are 0.  VEC:
// col + 8 <= cols or col >= cols, and the row is 16-byte aligned.  Otherwise at any alignment;
// a row's last, partial chunk is fetched as the last 8 elements of the row and moved into place
// by value(), so that it costs no access of its own.  Rows shorter than 8 go one by one.
template <class T, bool VEC>
struct Chunk8 {
  static constexpr bool HALF = sizeof(typename T::mem) == 2;
  u32x4_t u[HALF ? 1 : 2];
  __device__ __forceinline__ void load(const typename T::mem* row, long col, long cols) {
#pragma unroll
    for (int k = 0; k < (HALF ? 1 : 2); ++k) u[k] = u32x4_t{0u, 0u, 0u, 0u};
    if (col >= cols) return;
    if constexpr (VEC) {
#pragma unroll
      for (int k = 0; k < (HALF ? 1 : 2); ++k)
        u[k] = *reinterpret_cast<const u32x4_t*>(row + col + 4 * k);
    } else if (cols >= 8) {
      const typename T::mem* at = row + (col < cols - 8 ? col : cols - 8);
      if constexpr (HALF) {
        u[0] = *reinterpret_cast<const u32x4_a2*>(at);
      } else {
        u[0] = *reinterpret_cast<const u32x4_a4*>(at);
        u[1] = *reinterpret_cast<const u32x4_a4*>(at + 4);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i >= cols) break;
        if constexpr (HALF) u[0][i / 2] |= (uint32_t)row[i] << (16 * (i & 1));
        else u[i / 4][i & 3] = __float_as_uint(row[i]);
      }
    }
  }
  __device__ __forceinline__ void value(long col, long cols, float (&v)[8]) const {
    if constexpr (HALF) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(u[0][i]);
        v[2 * i + 1] = bf16_hi(u[0][i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i / 4][i & 3]);
    }
    if constexpr (!VEC) {
      const long over = col + 8 - cols;  // elements of the chunk past the row
      if (over > 0 && over < 8 && cols >= 8) {
#pragma unroll
        for (int bit = 4; bit > 0; bit /= 2)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] = (over & bit) ? (i + bit < 8 ? v[i + bit] : 0.f) : v[i];
      }
    }
  }
};

template <class T, bool VEC>
__device__ __forceinline__ void load8(const typename T::mem* row, long col, long cols, float (&v)[8]) {
  Chunk8<T, VEC> c;
  c.load(row, col, cols);
  c.value(col, cols, v);
}

template <class T, bool VEC>
__device__ __forceinline__ void store8(typename T::mem* row, long col, long cols, const float (&v)[8]) {
  if constexpr (VEC) {
    if (col < cols) {
      if constexpr (sizeof(typename T::mem) == 2) {
        const u32x4_t u = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                           pack_bf16(v[6], v[7])};
        *reinterpret_cast<u32x4_t*>(row + col) = u;
      } else {
        const f32x4_t a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
        *reinterpret_cast<f32x4_t*>(row + col) = a;
        *reinterpret_cast<f32x4_t*>(row + col + 4) = b;
      }
    }
  } else if (col + 8 <= cols) {
    if constexpr (sizeof(typename T::mem) == 2) {
      *reinterpret_cast<u32x4_a2*>(row + col) = u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                        pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    } else {
      *reinterpret_cast<f32x4_a4*>(row + col) = f32x4_t{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4_a4*>(row + col + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < cols) row[col + i] = T::from_f32(v[i]);
  }
}

// The first n of 16 bytes' elements to any element's address: one access where all of them count.
template <class T>
__device__ __forceinline__ void store_entries(typename T::mem* to, u32x4_t d, int n) {
  constexpr int E = 16 / (int)sizeof(typename T::mem);
  if (n >= E) {
    if constexpr (E == 8) *reinterpret_cast<u32x4_a2*>(to) = d;
    else *reinterpret_cast<u32x4_a4*>(to) = d;
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < n) {
        if constexpr (E == 8) to[i] = (uint16_t)(d[i / 2] >> (16 * (i & 1)));
        else to[i] = __uint_as_float(d[i]);
      }
  }
}

// Largest of the quad's values.
__device__ __forceinline__ uint32_t quad_max(uint32_t a) {
  uint32_t b = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0xB1, 0xf, 0xf, true);
  a = a > b ? a : b;
  b = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x4E, 0xf, 0xf, true);
  return a > b ? a : b;
}

// Scale byte of the block whose quad holds v: the exponent of the largest magnitude less
// that of the format's largest value, one more where its mantissa is larger than the
// format's; 255 (not a number) for a block with an infinity or NaN.  Magnitudes are
// compared as integers, which orders NaNs above everything.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(const float (&v)[8]) {
  constexpr int EMAX = FMT == kMxFp4 ? 2 : FMT == kMxFp8 ? 8 : 0;
  constexpr uint32_t MANT = FMT == kMxFp4 ? 0x400000u : FMT == kMxFp8 ? 0x600000u : 0x7e0000u;
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
    a = a > b ? a : b;
  }
  a = quad_max(a);
  const int ex = (int)(a >> 23);
  // a subnormal's leading bit is part of its mantissa: twice the limit's fraction
  const uint32_t lim = FMT == kMxInt8 && ex == 0 ? 0x7f0000u : MANT;
  const int e = ex - EMAX + ((a & 0x7fffffu) > lim ? 1 : 0);
  return ex == 255 ? 255u : (uint32_t)(e < 0 ? 0 : e > 254 ? 254 : e);
}

// 2^(127 - byte), 0 for byte 255.
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) {
  return __uint_as_float(byte < 254u ? (254u - byte) << 23 : byte == 254u ? 0x00400000u : 0u);
}
// 2^(byte - 127), NaN for byte 255.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23);
}

// d 2^(a - 127) 2^(b - 127), rounded once: neither scale on its own takes d past fp32's range.
__device__ __forceinline__ float mx_scale_product(float d, uint32_t a, uint32_t b) {
  const float v = __builtin_amdgcn_ldexpf(d, (int)(a + b) - 254);
  return a == 255u || b == 255u ? __uint_as_float(0x7fc00000u) : v;
}

// Codes of 8 elements over a scale: 4 bytes (fp4, even element in a byte's low half) or 8.
template <int FMT>
__device__ __forceinline__ u32x2_t mx_encode(const float (&v)[8], uint32_t byte) {
  const float inv = mx_inv_scale(byte);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = byte == 255u ? 0.f : v[i] * inv;
  u32x2_t r = {0u, 0u};
  if constexpr (FMT == kMxFp4) {
    r.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r.x, q[0], q[1], 1.0f, 0);
    r.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r.x, q[2], q[3], 1.0f, 1);
    r.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r.x, q[4], q[5], 1.0f, 2);
    r.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r.x, q[6], q[7], 1.0f, 3);
  } else if constexpr (FMT == kMxFp8) {
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
    r.x = (uint32_t)lo;
    r.y = (uint32_t)hi;
  } else {
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      // past 127 only where the scale has reached 2^127
      c[i] = (uint32_t)(int)fminf(fmaxf(rintf(q[i] * 64.f), -127.f), 127.f) & 255u;
    r.x = c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24);
    r.y = c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24);
  }
  return r;
}

// The values of 8 codes (fp4: r.x alone).
template <int FMT>
__device__ __forceinline__ void mx_decode(u32x2_t r, uint32_t byte, float (&v)[8]) {
  const float s = mx_scale(byte);
  if constexpr (FMT == kMxFp4) {
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.x, 1.0f, 0);
    const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.x, 1.0f, 1);
    const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.x, 1.0f, 2);
    const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r.x, 1.0f, 3);
    v[0] = a.x * s;
    v[1] = a.y * s;
    v[2] = b.x * s;
    v[3] = b.y * s;
    v[4] = c.x * s;
    v[5] = c.y * s;
    v[6] = d.x * s;
    v[7] = d.y * s;
  } else if constexpr (FMT == kMxFp8) {
    const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)r.x, false);
    const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)r.x, true);
    const f32x2_t c = __builtin_amdgcn_cvt_pk_f32_fp8((int)r.y, false);
    const f32x2_t d = __builtin_amdgcn_cvt_pk_f32_fp8((int)r.y, true);
    v[0] = a.x * s;
    v[1] = a.y * s;
    v[2] = b.x * s;
    v[3] = b.y * s;
    v[4] = c.x * s;
    v[5] = c.y * s;
    v[6] = d.x * s;
    v[7] = d.y * s;
  } else {
    // the code is the value times 64; 2^-6 first, so that a product near the smallest
    // scale is rounded once, by the last multiplication (it is exact there too)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = (float)(int8_t)(r.x >> (8 * i)) * 0.015625f * s;
      v[4 + i] = (float)(int8_t)(r.y >> (8 * i)) * 0.015625f * s;
    }
  }
}

}  // namespace flce
