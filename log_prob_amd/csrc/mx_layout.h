// Element types, microscaled formats and the bytes of their rows, for host and device code.
#pragma once

#include <stdint.h>

namespace flce {

// Element types and microscaled formats: the values of the C ABI's enumerations.
constexpr int kBf16 = 0, kF32 = 1;
constexpr int kMxNone = -1, kMxFp4 = 0, kMxFp8 = 1, kMxInt8 = 2;

// Microscaled layout: row bytes of codes (whole blocks of 32) and of scales (a multiple of
// 16, so that a row's scales can be read 16 bytes at a time).
constexpr int64_t mx_blocks(int64_t cols) { return (cols + 31) / 32; }
constexpr int64_t mx_code_bytes(int64_t cols, int fmt) {
  return mx_blocks(cols) * (fmt == kMxFp4 ? 16 : 32);
}
constexpr int64_t mx_scale_bytes(int64_t cols) { return (mx_blocks(cols) + 15) / 16 * 16; }

}  // namespace flce
