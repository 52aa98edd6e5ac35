// Quantisation to microscaled formats and back (gfx950): one pass, bound by memory.
//
//   quantise    codes = round(x / 2^e) with 2^e the block's scale; scale byte e + 127
//   dequantise  x = code 2^e
//
// A thread takes 8 consecutive elements at a time (a 16-byte load of bf16), so the block's
// scale is found by the four lanes of a quad and nothing goes through LDS.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "ops_internal.h"

namespace flce {

namespace {

constexpr int THREADS = 256;
constexpr int BATCH = 4;  // chunks a thread has in flight

// Offset of a row's scale bytes, and of block b's byte from there.
__device__ __forceinline__ long row_at(const MxScaleLayout& l, long row) {
  return (row >> 8) * l.tile_stride + (row & 255) * l.row_stride;
}
__device__ __forceinline__ long scale_at(const MxScaleLayout& l, long b) {
  return (b >> 4) * l.quad_stride + (b & 15);
}

// 16-byte pieces from [rows][quads] to [rows / 256][quads][256]: 8 lanes read 128 contiguous
// bytes of a row and 8 write 128 of a quad.
__device__ __forceinline__ void turn_scales(const MxTurn& p, unsigned group) {
  const u32x4_t* src = reinterpret_cast<const u32x4_t*>(p.src);
  u32x4_t* dst = reinterpret_cast<u32x4_t*>(p.dst);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, qtiles = (p.quads + 7) / 8;
  const long n = (p.rows + 7) / 8 * qtiles;
  for (long i = (long)group * (THREADS / 64) + wave; i < n; i += (long)p.groups * (THREADS / 64)) {
    const long row = i / qtiles * 8 + lane / 8;
    const int q = (int)(i % qtiles) * 8 + (lane & 7);
    if (row < p.rows && q < p.quads)
      dst[(row >> 8) * (256l * p.quads) + q * 256l + (row & 255)] = src[row * p.quads + q];
  }
}

// Rows of TPR threads, THREADS / TPR rows a workgroup; thread t of a row takes chunks t,
// t + TPR, ... of it.  A row's codes end with a whole block, so quads stay whole.
template <class T, int FMT, bool VEC>
__global__ __launch_bounds__(THREADS) void mx_quantize_kernel(MxQuantArgs p, int tpr) {
  if (p.clear && blockIdx.x == 0 && threadIdx.x < 8)
    __hip_atomic_store(&p.clear[threadIdx.x], 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const unsigned groups = gridDim.x - p.turn.groups;
  if (blockIdx.x >= groups) return turn_scales(p.turn, blockIdx.x - groups);
  const int t = threadIdx.x & (tpr - 1), rows = THREADS / tpr;
  const long blocks = mx_blocks(p.cols), chunks = 4 * blocks;
  const long code_ld = mx_code_bytes(p.cols, FMT), quads = mx_scale_bytes(p.cols) / 16;
  for (long row = (long)blockIdx.x * rows + threadIdx.x / tpr; row < p.rows; row += (long)groups * rows) {
    const typename T::mem* x = static_cast<const typename T::mem*>(p.x) + row * p.ldx;
    uint8_t* codes = p.codes + row * code_ld;
    uint8_t* scales = p.scales + row_at(p.layout, row);
    for (long c0 = t; c0 < chunks; c0 += (long)BATCH * tpr) {
      float v[BATCH][8];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) load8<T, VEC>(x, 8 * (c0 + (long)b * tpr), p.cols, v[b]);
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const long c = c0 + (long)b * tpr;
        if (c < chunks) {  // the same for a whole quad
          const uint32_t byte = mx_scale_byte<FMT>(v[b]);
          const u32x2_t q = mx_encode<FMT>(v[b], byte);
          if constexpr (FMT == kMxFp4)
            *reinterpret_cast<uint32_t*>(codes + 4 * c) = q.x;
          else
            *reinterpret_cast<u32x2_t*>(codes + 8 * c) = q;
          if ((c & 3) == 0) scales[scale_at(p.layout, c >> 2)] = (uint8_t)byte;
        }
      }
    }
    for (long i = blocks + t; i < 16 * quads; i += tpr) scales[scale_at(p.layout, i)] = 0;
  }
}

template <class T, int FMT, bool VEC>
__global__ __launch_bounds__(THREADS) void mx_dequantize_kernel(MxQuantArgs p, int tpr) {
  const int t = threadIdx.x & (tpr - 1), rows = THREADS / tpr;
  const long chunks = 4 * mx_blocks(p.cols);
  const long code_ld = mx_code_bytes(p.cols, FMT);
  for (long row = (long)blockIdx.x * rows + threadIdx.x / tpr; row < p.rows; row += (long)gridDim.x * rows) {
    typename T::mem* out = static_cast<typename T::mem*>(p.out) + row * p.ldo;
    const uint8_t* codes = p.codes + row * code_ld;
    const uint8_t* scales = p.scales + row_at(p.layout, row);
#pragma unroll 4
    for (long c = t; c < chunks; c += tpr) {
      u32x2_t q = {0u, 0u};
      if constexpr (FMT == kMxFp4)
        q.x = *reinterpret_cast<const uint32_t*>(codes + 4 * c);
      else
        q = *reinterpret_cast<const u32x2_t*>(codes + 8 * c);
      float v[8];
      mx_decode<FMT>(q, scales[scale_at(p.layout, c >> 2)], v);
      store8<T, VEC>(out, 8 * c, p.cols, v);
    }
  }
}

// Threads a row (a power of two, at least a quad): one chunk each in a small matrix, four in a
// large one, whose loads are then in flight together (128256 x 4096: 299 us with one or two,
// 258 us with four; 1 x 4096 and 64 x 4096 gain nothing from fewer threads).
int threads_per_row(long rows, long cols) {
  const long chunks = 4 * mx_blocks(cols);
  const long each = rows * chunks > (1l << 17) ? BATCH : 1;
  int t = 4;
  while (t < THREADS && t * each < chunks) t *= 2;
  return t;
}

// Workgroups stay and walk the rows (128256 x 4096 bf16 to MXFP4: 361 us with one a row, 282
// us with 16 a compute unit; back: 251 and 256 us with 32, but 151936 x 2048 201 and 160 us).
unsigned grid_of(const MxQuantArgs& a, int tpr, long most) {
  const long rows = THREADS / tpr, need = (a.rows + rows - 1) / rows;
  return (unsigned)(need < most ? need : most);
}

template <class T, int FMT, bool VEC>
void quantize(const MxQuantArgs& a, hipStream_t s) {
  const int tpr = threads_per_row(a.rows, a.cols);
  mx_quantize_kernel<T, FMT, VEC><<<grid_of(a, tpr, 16 * 256) + a.turn.groups, THREADS, 0, s>>>(a, tpr);
}
template <class T, int FMT, bool VEC>
void dequantize(const MxQuantArgs& a, hipStream_t s) {
  const int tpr = threads_per_row(a.rows, a.cols);
  mx_dequantize_kernel<T, FMT, VEC><<<grid_of(a, tpr, 32 * 256), THREADS, 0, s>>>(a, tpr);
}

template <int FMT>
void quantize_any(const MxQuantArgs& a, int dtype, bool vec, hipStream_t s) {
  if (dtype == kBf16) vec ? quantize<Bf16, FMT, true>(a, s) : quantize<Bf16, FMT, false>(a, s);
  else vec ? quantize<F32, FMT, true>(a, s) : quantize<F32, FMT, false>(a, s);
}
template <int FMT>
void dequantize_any(const MxQuantArgs& a, int dtype, bool vec, hipStream_t s) {
  if (dtype == kBf16) vec ? dequantize<Bf16, FMT, true>(a, s) : dequantize<Bf16, FMT, false>(a, s);
  else vec ? dequantize<F32, FMT, true>(a, s) : dequantize<F32, FMT, false>(a, s);
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs& a, int dtype, int fmt, bool vec, hipStream_t s) {
  if (fmt == kMxFp4) quantize_any<kMxFp4>(a, dtype, vec, s);
  else if (fmt == kMxFp8) quantize_any<kMxFp8>(a, dtype, vec, s);
  else quantize_any<kMxInt8>(a, dtype, vec, s);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxQuantArgs& a, int dtype, int fmt, bool vec, hipStream_t s) {
  if (fmt == kMxFp4) dequantize_any<kMxFp4>(a, dtype, vec, s);
  else if (fmt == kMxFp8) dequantize_any<kMxFp8>(a, dtype, vec, s);
  else dequantize_any<kMxInt8>(a, dtype, vec, s);
  return hipGetLastError();
}

}  // namespace flce
