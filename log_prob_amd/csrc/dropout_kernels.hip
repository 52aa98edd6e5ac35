// Dropout with a counter-based generator for gfx950, and the residual it is added to.
//
//   y = residual + x keep / (1 - q),   keep[m, h] = bits[m, h] >= threshold
//
// where q = threshold / 65536 and bits are 16 random bits of the element.  They come from
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3",
// SC11): the block with counter (h / 8, m, offset low, offset high) and key (seed low, seed
// high) serves 8 columns of a row, two a word.  The mask follows from the seed and the
// element's place alone, so it is never stored: the gradient is the same call on dy.
//
// A lane takes 8 columns, so a block of the generator is one lane's own: ten rounds of two
// 32 x 32 bit products.  With 32 bits an element it would cost twice that.  Sums and products
// are in fp32, rounded once at the store.
//
// Bound by memory: 32767 x 2048 bf16 with a residual 79 us (5.1 TB/s, the copy rate), without one
// 51.5 (5.2); four chunks a thread, loaded together, keep enough in flight.  65 x 1000 takes 2.7 us,
// the least that a launch takes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_internal.h"
#include "mx_device.h"

namespace flce {

namespace {

struct Words {
  uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                        uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

// A residual of either type, or none.
struct NoRes {};
template <class TR, bool VEC>
struct Residual {
  Chunk8<TR, VEC> c;
  __device__ __forceinline__ void load(const DropoutArgs& p, long row, int col) {
    c.load(static_cast<const typename TR::mem*>(p.residual) + row * p.ldr, col, p.H);
  }
  __device__ __forceinline__ void value(int col, int H, float (&v)[8]) const { c.value(col, H, v); }
};
template <bool VEC>
struct Residual<NoRes, VEC> {
  __device__ __forceinline__ void load(const DropoutArgs&, long, int) {}
  __device__ __forceinline__ void value(int, int, float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  }
};

// Chunks of 8 columns, row by row: a workgroup takes 256 U of them, thread t the chunks t, t +
// 256, ... of those, whose loads go out together.  `magic` is 2^42 / chunks of a row, rounded
// up: i * magic >> 42 is i / chunks for i < 2^21 (rows have at most 2^17 chunks).
template <class TX, class TR, class TY, bool VEC, int U>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs p, int chunks, uint64_t magic) {
  const uint64_t seed = p.seed_at ? *p.seed_at : p.seed;
  const uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
  const uint32_t o0 = (uint32_t)p.offset, o1 = (uint32_t)(p.offset >> 32);
  const long total = p.M * chunks;
  for (long first = (long)blockIdx.x * (256 * U); first < total; first += (long)gridDim.x * (256 * U)) {
    const long row0 = first / chunks;
    const uint32_t in0 = (uint32_t)(first - row0 * chunks) + threadIdx.x;
    Chunk8<TX, VEC> x[U];
    Residual<TR, VEC> res[U];
    long row[U];
    int col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = in0 + 256u * u, r = (uint32_t)((i * magic) >> 42);
      row[u] = row0 + r;
      // (a chunk past the last row has no columns)
      col[u] = row[u] < p.M ? 8 * (int)(i - r * (uint32_t)chunks) : p.H;
      if (row[u] >= p.M) row[u] = p.M - 1;
      x[u].load(static_cast<const typename TX::mem*>(p.x) + row[u] * p.ldx, col[u], p.H);
      res[u].load(p, row[u], col[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Words b = philox((uint32_t)col[u] >> 3, (uint32_t)row[u], o0, o1, k0, k1);
      float v[8], r[8];
      x[u].value(col[u], p.H, v);
      res[u].value(col[u], p.H, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t bits = i & 1 ? b.w[i / 2] >> 16 : b.w[i / 2] & 0xffffu;
        // (chosen, not multiplied by 0: a dropped infinity or NaN is gone)
        v[i] = bits >= p.threshold ? fmaf(v[i], p.up, r[i]) : r[i];
      }
      if (col[u] < p.H) store8<TY, VEC>(static_cast<typename TY::mem*>(p.y) + row[u] * p.ldy, col[u], p.H, v);
    }
  }
}

template <class TX, class TR, class TY>
void run(const DropoutArgs& a, bool vec, hipStream_t s) {
  const int chunks = (a.H + 7) / 8;
  const uint64_t magic = ((uint64_t(1) << 42) + uint64_t(chunks) - 1) / uint64_t(chunks);
  const long total = a.M * chunks;
  const long most = 1 << 22;  // workgroups; more work loops
  // few chunks: one a thread, so that every compute unit has some
  const long U = total > 256 * 1024 ? 4 : 1;
  const long need = (total + 256 * U - 1) / (256 * U);
  const unsigned grid = (unsigned)(need < most ? need : most);
  if (U == 4) {
    if (vec) dropout_kernel<TX, TR, TY, true, 4><<<grid, 256, 0, s>>>(a, chunks, magic);
    else dropout_kernel<TX, TR, TY, false, 4><<<grid, 256, 0, s>>>(a, chunks, magic);
  } else {
    if (vec) dropout_kernel<TX, TR, TY, true, 1><<<grid, 256, 0, s>>>(a, chunks, magic);
    else dropout_kernel<TX, TR, TY, false, 1><<<grid, 256, 0, s>>>(a, chunks, magic);
  }
}
template <class TX, class TY>
void with_residual(const DropoutArgs& a, int residual_dtype, bool vec, hipStream_t s) {
  if (residual_dtype == kNoResidual) run<TX, NoRes, TY>(a, vec, s);
  else if (residual_dtype == kF32) run<TX, F32, TY>(a, vec, s);
  else run<TX, Bf16, TY>(a, vec, s);
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, int x_dtype, int residual_dtype, int y_dtype, bool vec,
                          hipStream_t s) {
  if (x_dtype == kF32) {
    if (y_dtype == kF32) with_residual<F32, F32>(a, residual_dtype, vec, s);
    else with_residual<F32, Bf16>(a, residual_dtype, vec, s);
  } else {
    if (y_dtype == kF32) with_residual<Bf16, F32>(a, residual_dtype, vec, s);
    else with_residual<Bf16, Bf16>(a, residual_dtype, vec, s);
  }
  return hipGetLastError();
}

}  // namespace flce
