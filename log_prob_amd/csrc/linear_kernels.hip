// Matrix product with bias, activation and residual in its epilogue, and its gradient (gfx950).
//
//   pre = X W^T + bias,  y = act(pre) + residual
//   dpre = dy act'(pre),  dX = dpre W,  dW = dpre^T X,  dbias = sum_m dpre
//
// Products run on the bf16 MFMA mainloop of the head, whose operands may have their K contiguous
// or their rows, so no operand is transposed.  The accumulators leave through a slice of LDS of
// each wave's own, from which a lane takes 8 consecutive columns of a row: bias, activation and
// residual are applied there in fp32, and everything is read and written in 16-byte pieces.
//
// The rate of the matrix pipe bounds large products, the bytes of W small ones.  Tiles are
// 256 x 256 where they fill the chip, smaller ones (two or three workgroups a compute unit)
// otherwise; a long K over few tiles is split, the fp32 partial products added in order by a
// second kernel.  A decoding step (up to 32 rows) has kernels of its own that stream W.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "block_internal.h"
#include "mainloop_device.h"
#include "mx_device.h"
#include "tile_device.h"

namespace flce {

namespace {

// ---------------------------------------------------------------------------
// Activations in fp32.

// Phi(-z) e^(z^2 / 2) for z >= 0, Phi being the normal distribution: a polynomial in 1 / (1 +
// 0.3 z), fitted to the scaled complementary error function on [0, 15] for the least relative
// error (6e-8; 4e-7 with fp32 arithmetic).  The library's erff takes twice as long.  The exponentials
// beside it and in the logistic function are 2^y of an argument rounded to fp32: far in the tail, where
// y is -100, they are off by some 1e-5 of values below 1e-30.
__device__ __forceinline__ float scaled_tail(float z) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3f, z, 1.f));
  float p = 0.03842540085315704f;
  p = fmaf(p, t, -0.16939479112625122f);
  p = fmaf(p, t, 0.22913166880607605f);
  p = fmaf(p, t, -0.07704470306634903f);
  p = fmaf(p, t, 0.1429063081741333f);
  p = fmaf(p, t, 0.09452608972787857f);
  p = fmaf(p, t, 0.12196046113967896f);
  p = fmaf(p, t, 0.11948209255933762f);
  return fmaf(p, t, 7.495441423088778e-06f);
}
// Phi(x) and e^(-x^2 / 2).
__device__ __forceinline__ float normal_cdf(float x, float& ex) {
  ex = __builtin_amdgcn_exp2f(x * x * (-0.5f * LOG2E));
  const float q = scaled_tail(fabsf(x)) * ex;
  return x >= 0.f ? 1.f - q : q;  // (a NaN: q is one)
}
__device__ __forceinline__ float logistic(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-LOG2E * x));
}
constexpr float TANH_SCALE = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float TANH_CUBE = 0.044715f;

template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == kActRelu) return x < 0.f ? 0.f : x;
  float ex;
  if constexpr (ACT == kActGelu) return x * normal_cdf(x, ex);
  // (1 + tanh u) / 2 is the logistic function of 2 u
  if constexpr (ACT == kActGeluTanh) return x * logistic(TANH_SCALE * x * fmaf(TANH_CUBE * x, x, 1.f));
  if constexpr (ACT == kActSilu) return x * logistic(x);
  return x;
}
// f(integral_constant of act): the branch is the same for every lane.
template <class F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>()); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>()); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>()); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>()); break;
    default: f(std::integral_constant<int, kActNone>()); break;
  }
}
__device__ __forceinline__ float slope(float x, int act) {
  switch (act) {
    case kActRelu: return x > 0.f ? 1.f : x <= 0.f ? 0.f : x;
    case kActGelu: {
      float ex;
      const float cdf = normal_cdf(x, ex);
      return fmaf(x * 0.3989422804014327f, ex, cdf);
    }
    case kActGeluTanh: {
      // (beyond 30 the slope is 0 or 1, but x^2 may not be a number)
      const float z = x > 30.f ? 30.f : x < -30.f ? -30.f : x;
      const float s = logistic(TANH_SCALE * z * fmaf(TANH_CUBE * z, z, 1.f));
      return fmaf(z * s * (1.f - s), TANH_SCALE * fmaf(3.f * TANH_CUBE * z, z, 1.f), s);
    }
    case kActSilu: {
      const float s = logistic(x);
      return fmaf(x * s, 1.f - s, s);
    }
    default: return 1.f;
  }
}
__device__ __forceinline__ void activate8(float (&v)[8], int act) {
  with_act(act, [&](auto a) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = activate<decltype(a)::value>(v[i]);
  });
}

// ---------------------------------------------------------------------------
// The epilogue of 8 consecutive columns of a row.

// 8 elements of either type, as they come from memory.
struct AnyChunk {
  u32x4_t u[2];
  __device__ __forceinline__ void load(const void* p, int dtype, long at, int col, int cols) {
    if (dtype == kF32) {
      Chunk8<F32, false> c;
      c.load(static_cast<const float*>(p) + at, col, cols);
      u[0] = c.u[0];
      u[1] = c.u[1];
    } else {
      Chunk8<Bf16, false> c;
      c.load(static_cast<const uint16_t*>(p) + at, col, cols);
      u[0] = c.u[0];
    }
  }
  __device__ __forceinline__ void value(int dtype, int col, int cols, float (&v)[8]) const {
    if (dtype == kF32) {
      const Chunk8<F32, false> c{{u[0], u[1]}};
      c.value(col, cols, v);
    } else {
      const Chunk8<Bf16, false> c{{u[0]}};
      c.value(col, cols, v);
    }
  }
};
__device__ __forceinline__ void add8(float (&v)[8], const void* p, int dtype, long at, int col, int cols) {
  AnyChunk c;
  c.load(p, dtype, at, col, cols);
  float b[8];
  c.value(dtype, col, cols, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += b[i];
}
__device__ __forceinline__ void store_any(void* p, int dtype, long at, int col, int cols, const float (&v)[8]) {
  if (dtype == kF32) store8<F32, false>(static_cast<float*>(p) + at, col, cols, v);
  else store8<Bf16, false>(static_cast<uint16_t*>(p) + at, col, cols, v);
}
// The same with bf16 past the caches: a tile's results are not read again by its launch, and
// would push operands out of L2 (4096 x 4096 x 4096 with a bias: 107 -> 104.5 us, gelu 115 -> 113.5,
// with residual and pre too 149 -> 138).  fp32 stays in them (112 us against 134): its two stores a
// thread cover every other 16 bytes, and only the cache puts them together.
__device__ __forceinline__ void stream_any(void* p, int dtype, long at, int col, int cols, const float (&v)[8]) {
  if (dtype == kF32 || col + 8 > cols) return store_any(p, dtype, at, col, cols, v);
  const u32x4_a2 u = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  __builtin_nontemporal_store(u, reinterpret_cast<u32x4_a2*>(static_cast<uint16_t*>(p) + at + col));
}
__device__ __forceinline__ void finish8(const LinearEpilogue& e, long m, int col, int N, float (&v)[8]) {
  if (e.bias) add8(v, e.bias, e.bias_dtype, 0, col, N);
  if (e.pre) store8<Bf16, false>(e.pre + m * e.ldp, col, N, v);
  activate8(v, e.act);
  if (e.residual) add8(v, e.residual, e.residual_dtype, m * e.ldr, col, N);
  store_any(e.out, e.out_dtype, m * e.ldo, col, N, v);
}

// A wave's accumulators (WM x WN of the tile at (m0, n0)) to the epilogue, 64 rows at a time
// through its own slice of LDS: row r, column c at float r WN + (c ^ 32 ((r >> 2) & 1)), so that
// the two half-waves of a write (rows r and r + 4) meet different banks where rows are 64 columns
// or more.  A lane then has the same 8 columns of every row, and goes over the slice twice: bias,
// pre and activation in place, then the residual and the store.  The residual's loads go out half a
// slice at once, the first half ahead of everything else.
template <class S>
struct Slice {
  static constexpr int WN = S::WN, ROWS = 64, BLOCKS = ROWS / 32, COLS8 = WN / 8, PER = 64 / COLS8;
  static constexpr int STEPS = ROWS / PER, HALF = STEPS / 2;
  static constexpr int BYTES = S::NWAVES * ROWS * WN * 4;
  static_assert(S::MB % BLOCKS == 0, "slices");
  float* sl;
  int lane, row0;  // the slice's first row in D
  __device__ __forceinline__ int row(int it) const { return PER * it + lane / COLS8; }
  __device__ __forceinline__ float* at(int it) const {
    const int r = row(it);
    return sl + r * WN + ((8 * (lane % COLS8)) ^ (WN >= 64 ? ((r >> 2) & 1) << 5 : 0));
  }
  __device__ __forceinline__ void get(int it, float (&v)[8]) const {
    const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(at(it)), up = *reinterpret_cast<const f32x4_t*>(at(it) + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = lo[i];
      v[4 + i] = up[i];
    }
  }
  __device__ __forceinline__ void put(int it, const float (&v)[8]) const {
    *reinterpret_cast<f32x4_t*>(at(it)) = f32x4_t{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4_t*>(at(it) + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
  }
};

// FULL: with bias, pre, activation and residual, if any; otherwise (the gradients' products) the
// values go out as they are.  With `part` (a share of a split K) they go there in fp32.
template <class S, bool FULL>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[S::MB][S::NB], char* smem, const LinearEpilogue& e,
                                           float* part, long ldpart, int M, int N, int m0, int n0) {
  using L = Slice<S>;
  constexpr int WN = S::WN, HALF = L::HALF;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  L sl;
  sl.sl = reinterpret_cast<float*>(smem) + wave * L::ROWS * WN;
  sl.lane = lane;
  const int lc = lane & 31, hi = lane >> 5, sw = WN >= 64 ? hi << 5 : 0;
  const int col = n0 + (wave % S::WAVES_N) * WN + 8 * (lane % L::COLS8);
  const bool first_pass = FULL && !part && (e.bias || e.pre || e.act != kActNone);
  const bool residual = FULL && !part && e.residual;
  void* const to = part ? static_cast<void*>(part) : e.out;
  const int dtype = part ? kF32 : e.out_dtype;
  const long ld = part ? ldpart : e.ldo;
  float b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = 0.f;
  if (first_pass && e.bias) add8(b, e.bias, e.bias_dtype, 0, col, N);
  auto slice = [&](auto number) {
    constexpr int s = decltype(number)::value;
    sl.row0 = m0 + (wave / S::WAVES_N) * S::WM + L::ROWS * s;
    AnyChunk res[HALF];
    auto load_residual = [&](int it) {
      const int m = sl.row0 + sl.row(it);
      res[it % HALF].load(e.residual, e.residual_dtype, (long)m * e.ldr, col, m < M ? N : 0);
    };
    if (residual) {
#pragma unroll
      for (int i = 0; i < HALF; ++i) load_residual(i);
    }
#pragma unroll
    for (int mi = 0; mi < L::BLOCKS; ++mi)
#pragma unroll
      for (int nb = 0; nb < S::NB; ++nb)
#pragma unroll
        for (int q = 0; q < 16; ++q)
          sl.sl[(32 * mi + acc_row(lane, q)) * WN + ((32 * nb + lc) ^ sw)] = acc_read(acc[L::BLOCKS * s + mi][nb][q]);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (first_pass)
      with_act(e.act, [&](auto a) {
#pragma unroll 4
        for (int it = 0; it < L::STEPS; ++it) {
          const int m = sl.row0 + sl.row(it);
          float v[8];
          sl.get(it, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += b[i];
          if (e.pre && m < M) stream_any(e.pre, kBf16, (long)m * e.ldp, col, N, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = activate<decltype(a)::value>(v[i]);
          sl.put(it, v);
        }
      });
    if (residual) {
#pragma unroll
      for (int it = 0; it < L::STEPS; ++it) {
        const int m = sl.row0 + sl.row(it);
        float v[8], r[8];
        sl.get(it, v);
        res[it % HALF].value(e.residual_dtype, col, N, r);
        if (it < HALF) load_residual(it + HALF);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += r[j];
        if (m < M) stream_any(to, dtype, (long)m * ld, col, N, v);
      }
    } else {
#pragma unroll 4
      for (int it = 0; it < L::STEPS; ++it) {
        const int m = sl.row0 + sl.row(it);
        float v[8];
        sl.get(it, v);
        if (m < M) stream_any(to, dtype, (long)m * ld, col, N, v);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
  // (one after the other by name: a loop this long is not unrolled, and accumulators indexed at
  // run time would go to memory)
  slice(std::integral_constant<int, 0>());
  if constexpr (S::MB / L::BLOCKS == 2) slice(std::integral_constant<int, 1>());
  static_assert(S::MB / L::BLOCKS <= 2, "slices");
}

// The tile at (m0, n0) and share `split` of K.
template <class S, bool A_KC, bool B_KC>
__device__ __forceinline__ void product_tile(char* smem, int m0, int n0, int split, const LinearProduct& p,
                                             const LinearEpilogue& e, float* part, const LinearPlan& plan) {
  const int k0 = split * plan.k_each, k1 = min(p.K, k0 + plan.k_each);
  const TileSrc A{A_KC ? p.a + (long)m0 * p.lda + k0 : p.a + (long)k0 * p.lda + m0, p.lda, p.M - m0,
                  min(p.kvalid_a, k1) - k0, 0};
  const TileSrc B{B_KC ? p.b + (long)n0 * p.ldb + k0 : p.b + (long)k0 * p.ldb + n0, p.ldb, p.N - n0,
                  min(p.kvalid_b, k1) - k0, 0};
  f32x16 acc[S::MB][S::NB];
  mainloop<S, A_KC, B_KC>(acc, smem, A, B, k1 - k0);
  const long ldpart = (p.N + 7) / 8 * 8;
  float* mine = plan.splits > 1 ? part + (long)split * p.M * ldpart : nullptr;
  store_tile<S, A_KC && B_KC>(acc, smem, e, mine, ldpart, p.M, p.N, m0, n0);
}

// Workgroup `id` of n_mt x n_nt tiles times `splits` shares of K.  Workgroups of one XCD take
// neighbouring tiles of the same share (groups of 8 tile rows).  The last tile row is one of the
// lower shape T where that holds it.
template <class S, class T, bool A_KC, bool B_KC>
__device__ __forceinline__ void run_tile(char* smem, int id, const LinearProduct& p, const LinearEpilogue& e,
                                         float* part, const LinearPlan& plan) {
  static_assert(T::TN == S::TN && T::PIPE_BYTES <= S::PIPE_BYTES && T::NTHREADS == S::NTHREADS, "lower shape");
  static_assert(Slice<S>::BYTES <= S::PIPE_BYTES && Slice<T>::BYTES <= S::PIPE_BYTES, "slices");
  const int n_mt = (p.M + S::TM - 1) / S::TM, n_nt = (p.N + S::TN - 1) / S::TN;
  const int tiles = n_mt * n_nt, per = tiles * plan.splits >> 3;
  const int L = id < (per << 3) ? (id & 7) * per + (id >> 3) : id;
  const int split = L / tiles;
  int mt, nt;
  group_coords(L - split * tiles, n_mt, n_nt, 8, mt, nt);
  const int m0 = mt * S::TM, n0 = nt * S::TN;
  if constexpr (T::TM < S::TM) {
    if (p.M - m0 <= T::TM) return product_tile<T, A_KC, B_KC>(smem, m0, n0, split, p, e, part, plan);
  }
  product_tile<S, A_KC, B_KC>(smem, m0, n0, split, p, e, part, plan);
}

using Tile128 = Shape<128, 128, 64, 2, 2>;
using Tile64 = Shape<64, 128, 64, 2, 2, 1, 4>;
template <class S>
using Lower = std::conditional_t<S::TM == 256, Shape<128, 256, 64, 2, 1>, Tile64>;

template <class S>
__global__ __launch_bounds__(S::NTHREADS, S::WAVES_PER_EU) void linear_tile_kernel(LinearProduct p, LinearEpilogue e,
                                                                                  float* part, LinearPlan plan) {
  __shared__ __attribute__((aligned(1024))) char smem[S::PIPE_BYTES];
  run_tile<S, Lower<S>, true, true>(smem, blockIdx.x, p, e, part, plan);
}

// The partial products of a split K, added in order, and the epilogue: 8 columns a thread.
__global__ __launch_bounds__(256) void linear_join_kernel(LinearEpilogue e, const float* part, long ldpart,
                                                          int splits, long M, int N) {
  const int chunks = (N + 7) / 8;
  const long total = M * chunks;
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long)gridDim.x * 256) {
    const long m = i / chunks;
    const int col = 8 * (int)(i - m * chunks);
    const float* from = part + m * ldpart + col;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(from + s * M * ldpart);
      const f32x4_t up = *reinterpret_cast<const f32x4_t*>(from + s * M * ldpart + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] += lo[j];
        v[4 + j] += up[j];
      }
    }
    finish8(e, m, col, N, v);
  }
}

// ---------------------------------------------------------------------------
// One or two (MT) rows of X: W is read once, and bounds the call.  A wave takes R rows of W, its
// lanes 8 consecutive K each (1 KiB of a row at once), in batches of U loads a row; the next
// batch is in flight under the work on this one.  X lies in LDS, at most 64 KiB of it at a time,
// staged under the first batch, and is read from there once for the R rows.  Products of a pair of
// bf16 go through v_dot2: two multiplications and no unpacking.  1 x 4096 x 4096 8.6 us among other
// calls (3.9 TB/s; 9.9 alone, of which 2.5 are the launch's), 1 x 50257 x 1600 25.5 (6.3 TB/s); R of 1
// or 4 and U of 1 or 4 are up to 20% slower on one or the other.
__device__ __forceinline__ float load1(const void* p, int dtype, long at) {
  return dtype == kF32 ? static_cast<const float*>(p)[at] : Bf16::to_f32(static_cast<const uint16_t*>(p)[at]);
}
// The epilogue of one element.
__device__ __forceinline__ void finish1(const LinearEpilogue& e, long m, int n, float v) {
  if (e.bias) v += load1(e.bias, e.bias_dtype, n);
  if (e.pre) e.pre[m * e.ldp + n] = Bf16::from_f32(v);
  with_act(e.act, [&](auto a) { v = activate<decltype(a)::value>(v); });
  if (e.residual) v += load1(e.residual, e.residual_dtype, m * e.ldr + n);
  if (e.out_dtype == kF32) static_cast<float*>(e.out)[m * e.ldo + n] = v;
  else static_cast<uint16_t*>(e.out)[m * e.ldo + n] = Bf16::from_f32(v);
}

constexpr int FEW_LDS = 64 * 1024;
typedef float f32x4_acc __attribute__((ext_vector_type(4)));
constexpr int FEW_R = 2;
typedef __bf16 bf16x2_v __attribute__((ext_vector_type(2)));

template <int MT>
__global__ __launch_bounds__(256) void linear_few_kernel(LinearProduct p, LinearEpilogue e, int k_stage) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  constexpr int R = FEW_R, U = 2, NVAL = R * MT, BATCH = 512 * U;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  u32x4_t* xs = reinterpret_cast<u32x4_t*>(smem);  // [MT][k_stage / 8]
  const int groups = (p.N + 4 * R - 1) / (4 * R), ld8 = k_stage / 8;
  bool staged = false;
  for (int g = blockIdx.x; g < groups; g += gridDim.x) {
    const int n0 = (4 * g + wave) * R;
    float acc[NVAL];
#pragma unroll
    for (int i = 0; i < NVAL; ++i) acc[i] = 0.f;
    for (int ks = 0; ks < p.K; ks += k_stage) {
      const int len = min(k_stage, p.K - ks);
      const uint16_t* w[R];
#pragma unroll
      for (int r = 0; r < R; ++r) w[r] = p.b + (long)min(n0 + r, p.N - 1) * p.ldb + ks + 8 * lane;
      u32x4_t wv[2][U][R];
      auto load = [&](int b, int k0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int r = 0; r < R; ++r)
            wv[b][u][r] = k0 + 512 * u + 8 * lane < len
                              ? __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(w[r] + k0 + 512 * u))
                              : zero;
      };
      auto use = [&](int b, int k0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = k0 + 512 * u + 8 * lane;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const u32x4_t x = k < len ? xs[m * ld8 + k / 8] : zero;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                // (values of their own: a cast of a vector's element takes the vector's first)
                const uint32_t wi = wv[b][u][r][i], xi = x[i];
                acc[r * MT + m] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_v, wi),
                                                                  __builtin_bit_cast(bf16x2_v, xi),
                                                                  acc[r * MT + m], false);
              }
          }
        }
      };
      load(0, 0);
      if (!staged) {
        __syncthreads();
        for (int m = 0; m < MT; ++m)
          for (int c = threadIdx.x; c < len / 8; c += 256)
            xs[m * ld8 + c] = m < p.M ? *reinterpret_cast<const u32x4_t*>(p.a + m * p.lda + ks + 8 * c) : zero;
        __syncthreads();
        staged = k_stage >= p.K;
      }
      for (int k = 0; k < len; k += 2 * BATCH) {
        load(1, k + BATCH);
        use(0, k);
        load(0, k + 2 * BATCH);
        use(1, k + BATCH);
      }
    }
    // the sums over the lanes: each exchange halves the values a lane holds, so that in the end
    // lane l has the whole sum of one, and its 64 / NVAL neighbours the same
    int which = 0, off = 32;
#pragma unroll
    for (int n = NVAL; n > 1; n /= 2) {
      const bool up = lane & off;
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        const float keep = up ? acc[i + n / 2] : acc[i], give = up ? acc[i] : acc[i + n / 2];
        acc[i] = keep + __shfl_xor(give, off);
      }
      which += up ? n / 2 : 0;
      off /= 2;
    }
    float v = acc[0];
    for (; off > 0; off /= 2) v += __shfl_xor(v, off);
    const int r = which / MT, m = which % MT, n = n0 + r;
    if ((lane & (64 / NVAL - 1)) == 0 && m < p.M && n < p.N) finish1(e, m, n, v);
  }
}

// Up to 16 MB rows of X on the matrix instruction (16 x 16 x 32): a workgroup takes 16 rows of W,
// 512 K a stage through a ring of LDS stages by direct-to-LDS loads of 1 KiB of one row each; its
// four waves multiply 128 K of a stage each, and the four partial products meet in LDS and are
// added in order.  X is staged beside W, from L2.  Chunk c (16 bytes) of row r lies at position c ^
// (r % 16) of the row's 64, so that the 16 rows a fragment read touches fall on all banks.  (Loaded
// straight into the instruction's operands, 64 bytes of 16 rows at once, 16 x 50257 x 1600 took 52 us.)
template <int MB>
struct StreamShape {
  static constexpr int W_BYTES = 16 * 1024, STAGE = W_BYTES + MB * 16 * 1024;
  static constexpr int NS = 3;                  // stages (4 and 5 no quicker, 2 slower by a fifth)
  static constexpr int LOADS = 4 + 4 * MB;      // of a wave for a stage
  static_assert(NS * STAGE <= 160 * 1024 && 4 * MB * 1024 <= NS * STAGE, "LDS");
};

template <int MB>
__global__ __launch_bounds__(256) void linear_stream_kernel(LinearProduct p, LinearEpilogue e) {
  using C = StreamShape<MB>;
  __shared__ __attribute__((aligned(1024))) char smem[C::NS * C::STAGE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4, n0 = 16 * (int)blockIdx.x;
  const int nk = (p.K + 511) / 512, wvalid = p.N - n0;
  const i32x4 wr = make_rsrc_fixed(p.b + (long)n0 * p.ldb), xr = make_rsrc_fixed(p.a);
  const uint32_t lds0 = lds_addr_of(smem), ldw = (uint32_t)p.ldb * 2u, ldx = (uint32_t)p.lda * 2u;
  auto issue = [&](int k, int slot) {
    const uint32_t st = lds0 + (uint32_t)(slot * C::STAGE);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * wave + i, c = 64 * k + (lane ^ row);
      const bool ok = row < wvalid && 8 * c < p.K;
      dma16<0>(wr, ok ? (uint32_t)row * ldw + 16u * (uint32_t)c : OOB_OFFSET, 0u, st + 1024u * (uint32_t)row);
    }
#pragma unroll
    for (int i = 0; i < 4 * MB; ++i) {
      const int row = 4 * MB * wave + i, c = 64 * k + (lane ^ (row & 15));
      const bool ok = row < p.M && 8 * c < p.K;
      dma16<0>(xr, ok ? (uint32_t)row * ldx + 16u * (uint32_t)c : OOB_OFFSET, 0u,
               st + (uint32_t)C::W_BYTES + 1024u * (uint32_t)row);
    }
  };
  f32x4_acc acc[MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) acc[mb] = f32x4_acc{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < C::NS - 1; ++k) issue(k, k);
  int slot = 0;
  for (int k = 0; k < nk; ++k) {
    // stage k has landed, and every wave is done with stage k - 1, whose slot the next loads take
    // (steps past K only zero-fill it)
    wait_vmcnt<C::LOADS*(C::NS - 2)>();
    __syncthreads();
    issue(k + C::NS - 1, slot == 0 ? C::NS - 1 : slot - 1);
    const char* st = smem + slot * C::STAGE;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = ((16 * wave + 4 * i + q) ^ r) << 4;
      const bf16x8 w = *reinterpret_cast<const bf16x8*>(st + 1024 * r + at);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const bf16x8 x = *reinterpret_cast<const bf16x8*>(st + C::W_BYTES + 1024 * (16 * mb + r) + at);
        acc[mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, acc[mb], 0, 0, 0);
      }
    }
    slot = slot == C::NS - 1 ? 0 : slot + 1;
  }
  // the zero fills past the end must land before the LDS is used again
  wait_vmcnt<0>();
  __syncthreads();
  // lane l, element j: row 4 (l / 16) + j of W, row l % 16 of X's block
  float(*red)[MB][256] = reinterpret_cast<float(*)[MB][256]>(smem);
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[wave][mb][(4 * q + j) * 16 + r] = acc[mb][j];
  __syncthreads();
  // neighbouring threads take neighbouring columns of a row of the result
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int m = 16 * mb + (int)threadIdx.x / 16, c = threadIdx.x % 16, at = c * 16 + (int)threadIdx.x / 16;
    const float v = ((red[0][mb][at] + red[1][mb][at]) + red[2][mb][at]) + red[3][mb][at];
    if (m < p.M && c < wvalid) finish1(e, m, n0 + c, v);
  }
}

// ---------------------------------------------------------------------------
// dpre = dy act'(pre), 8 columns a lane and 512 a workgroup, whose four waves walk the rows of
// its group; the column sums stay in registers and meet in LDS.
// Bound by memory (4096 x 4096 bf16 24.4 us, of 100 MB; 513 x 1000 fp32 7.2, one round of waits).
constexpr int SLOPE_COLS = 512, SLOPE_ROWS = 4;  // rows a wave has in flight

template <class TY, bool VEC>
__global__ __launch_bounds__(256) void linear_slope_kernel(LinearSlopeArgs p) {
  __shared__ float red[3][SLOPE_COLS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * SLOPE_COLS + 8 * lane;
  const long each = (p.M + p.groups - 1) / p.groups;
  const long r0 = blockIdx.y * each, r1 = r0 + each < p.M ? r0 + each : p.M;
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.f;
  for (long r = r0 + wave * SLOPE_ROWS; r < r1; r += 4 * SLOPE_ROWS) {
    Chunk8<TY, VEC> dy[SLOPE_ROWS];
    Chunk8<Bf16, VEC> pre[SLOPE_ROWS];
#pragma unroll
    for (int j = 0; j < SLOPE_ROWS; ++j) {
      const long cols = r + j < r1 ? p.N : 0;
      dy[j].load(static_cast<const typename TY::mem*>(p.dy) + (r + j) * p.lddy, col, cols);
      if (p.pre) pre[j].load(p.pre + (r + j) * p.ldp, col, cols);
    }
#pragma unroll
    for (int j = 0; j < SLOPE_ROWS; ++j) {
      float v[8];
      dy[j].value(col, p.N, v);
      if (p.pre) {
        float x[8];
        pre[j].value(col, p.N, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= slope(x[i], p.act);
      }
      if (r + j < r1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = col + i < p.N ? v[i] : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += v[i];
        if (p.dpre) store8<Bf16, true>(p.dpre + (r + j) * p.ldd, col, p.ldd, v);
      }
    }
  }
  if (!p.part) return;
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) red[wave - 1][8 * lane + i] = sum[i];
  }
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int w = 0; w < 3; ++w) sum[i] += red[w][8 * lane + i];
      if (col + i < p.N) p.part[(long)blockIdx.y * p.N + col + i] = sum[i];
    }
  }
}

// dX of up to 1024 values: dX[m] = sum_n dpre[m, n] W[n], with dpre in fp32.  The rounding to bf16
// that the matrix instruction asks for adds as much to dX as the store's own, 1.4 times together, on
// average; the fewer values, the further from that average (1 x 37832 x 104: 2.4 to 2.7e-3 of the
// norm, this way 1.6e-3).  dW, which has as many values as the layer, goes without.
// A workgroup takes 4 rows, 512 columns and a share of n, 128 of which have their dpre in LDS at a
// time; a wave's lanes lie along a row of W, several rows at once where K is short.  The lanes' sums
// meet by exchange, the waves' in LDS, the shares' in the joining kernel, in a fixed order.
// dX alone (us, this way and by tiles): 5 x 3000 x 200 11.9, 12.9; 16 x 50257 x 64 22.9, 26.5; 128 x
// 4096 x 8 11.8, 14.4; 1 x 37832 x 104 19.9, 20.5; 1 x 4096 x 1024 14.3, 12.8; 4 x 50257 x 256 40, 26;
// 1 x 50257 x 1024 66, 29 (20 for W's bytes at the copy rate): latency, at most 96 shares.  With dbias
// or dW beside it this way adds 4 to 10 us for launches that the tiles share.  For more values the tiles
// are right, and quicker by more (4 x 4096 x 4096 29 us against 43).
constexpr int DX_ROWS = 4, DX_STAGE = 128, DX_COLS = 512;
template <class TY>
__global__ __launch_bounds__(256) void linear_few_dx_kernel(LinearFewDx p) {
  __shared__ float d[DX_ROWS][DX_STAGE];
  __shared__ __attribute__((aligned(16))) float red[4][DX_ROWS][DX_COLS];
  const int tid = threadIdx.x, m0 = DX_ROWS * (int)blockIdx.z, col0 = blockIdx.x * DX_COLS, lanes = p.lanes;
  const int col = col0 + 8 * (tid & (lanes - 1)), sub = tid / lanes, subs = 256 / lanes;
  const int n0 = blockIdx.y * p.each, n1 = min(p.N, n0 + p.each);
  float acc[DX_ROWS][8];
#pragma unroll
  for (int m = 0; m < DX_ROWS; ++m)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[m][i] = 0.f;
  for (int base = n0; base < n1; base += DX_STAGE) {
    __syncthreads();
#pragma unroll
    for (int i = tid; i < DX_ROWS * DX_STAGE; i += 256) {
      const int m = m0 + i / DX_STAGE, n = base + i % DX_STAGE;
      float v = 0.f;
      if (m < p.M && n < n1) {
        v = TY::to_f32(static_cast<const typename TY::mem*>(p.dy)[m * p.lddy + n]);
        if (p.pre) v *= slope(Bf16::to_f32(p.pre[m * p.ldp + n]), p.act);
      }
      d[i / DX_STAGE][i % DX_STAGE] = v;
    }
    __syncthreads();
    const int here = min(DX_STAGE, n1 - base);
    if (col < p.K) {
#pragma unroll 8
      for (int j = sub; j < here; j += subs) {
        const u32x4_t u = *reinterpret_cast<const u32x4_t*>(p.w + (long)(base + j) * p.ldw + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float w = i & 1 ? bf16_hi(u[i / 2]) : bf16_lo(u[i / 2]);
#pragma unroll
          for (int m = 0; m < DX_ROWS; ++m) acc[m][i] = fmaf(d[m][j], w, acc[m][i]);
        }
      }
    }
  }
  // the rows of W that share a wave, then the waves in order
  for (int off = 32; off >= lanes; off >>= 1) {
#pragma unroll
    for (int m = 0; m < DX_ROWS; ++m)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[m][i] += __shfl_xor(acc[m][i], off);
  }
  if ((tid & 63) < lanes) {
#pragma unroll
    for (int m = 0; m < DX_ROWS; ++m)
#pragma unroll
      for (int i = 0; i < 8; ++i) red[tid >> 6][m][8 * (tid & 63) + i] = acc[m][i];
  }
  __syncthreads();
  const int m = m0 + tid / lanes;
  if (tid < DX_ROWS * lanes && m < p.M && col < p.K) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = 8 * (tid & (lanes - 1)) + i;
      v[i] = ((red[0][m - m0][c] + red[1][m - m0][c]) + red[2][m - m0][c]) + red[3][m - m0][c];
    }
    if (p.splits > 1) store_any(p.part, kF32, ((long)blockIdx.y * p.M + m) * p.K, col, p.K, v);
    else store_any(p.dx, kBf16, m * p.lddx, col, p.K, v);
  }
}

// The groups' column sums added in order: 32 columns a workgroup, 8 shares of the groups.
__device__ __forceinline__ void bias_sum(char* smem, int id, const LinearBiasSum& b) {
  float(*red)[32] = reinterpret_cast<float(*)[32]>(smem);
  const int c = threadIdx.x & 31, sl = threadIdx.x >> 5, col = id * 32 + c;
  float s = 0.f;
  if (col < b.N) {
#pragma unroll 4
    for (int g = sl; g < b.groups; g += 8) s += b.part[(long)g * b.N + col];
  }
  red[sl][c] = s;
  __syncthreads();
  if (sl == 0 && col < b.N) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += red[k][c];
    if (b.dtype == kF32) static_cast<float*>(b.dbias)[col] = s;
    else static_cast<uint16_t*>(b.dbias)[col] = Bf16::from_f32(s);
  }
}

// The whole gradient after dpre in one launch: the tiles of dX, those of dW and the bias sums,
// none of which depends on another (at 513 x 1000 x 2048, where neither product fills the chip,
// one after the other they took 31 us).
template <class SX, class SW>
__global__ __launch_bounds__(256, SX::WAVES_PER_EU) void linear_grad_kernel(LinearGradArgs p) {
  constexpr int LDS = SX::PIPE_BYTES > SW::PIPE_BYTES ? SX::PIPE_BYTES : SW::PIPE_BYTES;
  static_assert(SX::NTHREADS == 256 && SW::NTHREADS == 256 && SX::WAVES_PER_EU == SW::WAVES_PER_EU, "one launch");
  __shared__ __attribute__((aligned(1024))) char smem[LDS];
  int id = blockIdx.x;
  if (id < p.n_dw) {
    run_tile<SW, SW, false, false>(smem, id, p.dw, p.out_dw, p.part_dw, p.plan_dw);
    return;
  }
  id -= p.n_dw;
  if (id < p.n_dx) {
    run_tile<SX, SX, true, false>(smem, id, p.dx, p.out_dx, p.part_dx, p.plan_dx);
    return;
  }
  bias_sum(smem, id - p.n_dx, p.bias);
}

// ---------------------------------------------------------------------------

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A plan's time in us.  Workgroups go to the 256 compute units in turn, `resident` at once.  A step
// of 64 K takes (measured at K = 4096, the tiles of one, two and three a unit): 64 x 128 0.54,
// 0.64, 0.83 us; 128 x 128 0.60, 0.90; 256 x 256 1.05 with few units busy and 1.65 with all of them
// (the clock).  A launch adds 3, a split a second launch and its partial products there and back
// at the copy rate; the operands come at 4.4 TB/s at
// most.  E.g. (us; tile/splits):
//   64 x 4096 x 4096     64/8 14.7, 128/8 15.4, 256/8 22, 64/1 35
//   512 x 4096 x 4096    64/2 31, 128/2 32, 64/1 36, 256/4 40, 128/1 40
//   1024 x 4096 x 4096   64/1 42, 128/1 43, 256/4 54, 256/1 69
//   2048 x 4096 x 4096   128/1 62, 256/1 74, 64/1 87
//   4096 x 4096 x 4096   256/1 101, 128/1 113, 64/1 146
// Operands past about 100 MB come from memory in earnest, which slows the small tiles' steps more,
// as they load more for a product:
//   256 x 50257 x 1600   256/1 59, 128/1 79, 64/1 90
//   257 x 50257 x 1600   256/1 81, 128/1 81, 64/1 87; with fp32 results 90, 87, 91
//   1024 x 32768 x 2048  256/1 115, 128/1 165, 64/1 199
// (Other shapes of tiles: 128 x 128 with 32 K a stage and three workgroups a unit 10 to 30% slower
// than 128/1 throughout, 128 x 256 with one workgroup 2 to 30%.)  The results' bytes are not part of the
// model: it has 72 and 78 us for 256/1 and 128/1 at 257 rows and takes the former, also where fp32
// results make it the slower by 4%; and 109 for 4096 x 4096 x 4096, which the whole epilogue (gelu,
// residual, pre) makes 136 (128/1 150, 64/1 193).
//
// `lower`: the last tile row is half as high where that holds it, which the model has a unit take
// beside another tile for 0.12 us a step, alone for 0.5 (tiles of 256 0.9).  It saves the operand's
// traffic where the last tiles run beside others (us, full height and half: 257 x 50257 x 1600 fp32 tiles
// of 128 88, 85, of 256 93, 89; 300 x 50257 x 1600 92, 89 and 95, 89; 320 x 16384 x 4096 65, 64 and 70,
// 67), and nothing where they run alone, as each step waits for its loads (1025 and 4097 x 4096 x 4096,
// 2100 x 8192 x 2048).  The gradients' products, several of which share a launch, go without.
double plan_time(const LinearPlan& p, int64_t M, int64_t N, int64_t K, bool lower) {
  const int64_t columns = cdiv(N, p.tile_n) * p.splits, n = cdiv(M, p.tile_m) * columns;
  const int64_t over = M % p.tile_m;
  const int64_t low = lower && p.tile_m > 64 && over > 0 && over <= p.tile_m / 2 ? columns : 0;
  const double steps = double(cdiv(p.k_each, 64));
  const int resident = p.tile_m == 256 ? 1 : p.tile_m == 128 ? 2 : 3;
  const double full = double(n) / 256 < 1 ? double(n) / 256 : 1;
  auto step = [&](int r) {
    if (r == 0) return 0.0;
    if (p.tile_m == 256) return 1.05 + 0.6 * full * full;
    if (p.tile_m == 128) return r == 1 ? 0.60 : 0.90;
    return r == 1 ? 0.54 : r == 2 ? 0.64 : 0.83;
  };
  int64_t load = cdiv(n - low, 256), more = cdiv(n, 256) - load;  // tiles a unit, and lower ones
  if (load == 0) {
    load = more;
    more = 0;
  }
  double t = double(load / resident) * step(resident) + step(int(load % resident));
  t += double(more) * (p.tile_m == 256 ? 0.9 : load % resident ? 0.12 : 0.5);
  t *= steps;
  const double bytes = 2.0 * (double(M) * K + double(N) * K);
  if (bytes > 100e6) t *= p.tile_m == 256 ? 1.08 : p.tile_m == 128 ? 1.3 : 1.5;
  t += 3;
  if (t < bytes / 4.4e6) t = bytes / 4.4e6;
  if (p.splits > 1) t += 4.5 + 8.0 * p.splits * double(M) * double(N) / 5.0e6;
  return t;
}

LinearPlan plan_of(int tile, int64_t splits, int64_t K) {
  LinearPlan p{};
  p.tile_m = tile;
  p.tile_n = tile == 64 ? 128 : tile;
  const int64_t k = K > 0 ? K : 1;
  p.k_each = int(cdiv(cdiv(k, splits), 64) * 64);
  p.splits = int(cdiv(k, p.k_each));
  return p;
}
// The quickest plan among the tiles from `least` to `most` that a launch can hold (time 1e30, and the
// largest tiles, where none is).
LinearPlan best_plan(int64_t M, int64_t N, int64_t K, int least, int most, bool lower, double* time) {
  LinearPlan best = plan_of(most, 1, K);
  *time = 1e30;
  for (int tile = least; tile <= most; tile *= 2)
    for (int64_t splits : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
      if (splits > 1 && K / splits < 128) break;
      const LinearPlan p = plan_of(tile, splits, K);
      if (!linear_fits(p, M, N)) break;
      const double t = plan_time(p, M, N, K, lower);
      if (t < *time) {
        *time = t;
        best = p;
      }
    }
  return best;
}

hipError_t join(const LinearProduct& p, const LinearPlan& plan, const LinearEpilogue& e, const float* part,
                hipStream_t s) {
  const long total = (long)p.M * ((p.N + 7) / 8), need = (total + 255) / 256;
  const unsigned grid = (unsigned)(need < 4096 ? need : 4096);
  linear_join_kernel<<<grid, 256, 0, s>>>(e, part, linear_part_ld(p.N), plan.splits, p.M, p.N);
  return hipGetLastError();
}

}  // namespace

LinearPlan linear_forward_plan(int64_t M, int64_t N, int64_t K) {
  double t;
  return best_plan(M, N, K, 64, 256, true, &t);
}

void linear_backward_plans(int64_t M, int64_t N, int64_t K, LinearPlan* dx, LinearPlan* dw) {
  // both run in one launch: large tiles for both, or small ones (dW's operands are read by
  // columns, which takes tiles of 128 at least)
  double big_x, big_w, small_x, small_w;
  const LinearPlan bx = best_plan(M, K, N, 256, 256, false, &big_x), bw = best_plan(N, K, M, 256, 256, false, &big_w);
  const LinearPlan sx = best_plan(M, K, N, 64, 128, false, &small_x), sw = best_plan(N, K, M, 128, 128, false, &small_w);
  const bool big = big_x + big_w < small_x + small_w;
  *dx = big ? bx : sx;
  *dw = big ? bw : sw;
}

int64_t linear_workgroups(const LinearPlan& p, int64_t M, int64_t N) {
  return cdiv(M, p.tile_m) * cdiv(N, p.tile_n) * p.splits;
}

hipError_t launch_linear_product(const LinearProduct& p, const LinearPlan& plan, const LinearEpilogue& e, float* part,
                                 hipStream_t s) {
  const unsigned grid = (unsigned)linear_workgroups(plan, p.M, p.N);
  if (plan.tile_m == 256) linear_tile_kernel<BigShape><<<grid, BigShape::NTHREADS, 0, s>>>(p, e, part, plan);
  else if (plan.tile_m == 128) linear_tile_kernel<Tile128><<<grid, Tile128::NTHREADS, 0, s>>>(p, e, part, plan);
  else linear_tile_kernel<Tile64><<<grid, Tile64::NTHREADS, 0, s>>>(p, e, part, plan);
  const hipError_t err = hipGetLastError();
  return err != hipSuccess || plan.splits == 1 ? err : join(p, plan, e, part, s);
}

hipError_t launch_linear_grad(LinearGradArgs a, hipStream_t s) {
  const unsigned bias = a.bias.dbias ? (unsigned)((a.bias.N + 31) / 32) : 0u;
  const unsigned grid = (unsigned)a.n_dx + (unsigned)a.n_dw + bias;
  if (grid == 0) return hipSuccess;
  if (a.plan_dw.tile_m == 256) linear_grad_kernel<BigShape, BigShape><<<grid, 256, 0, s>>>(a);
  else if (a.plan_dx.tile_m == 128) linear_grad_kernel<Tile128, Tile128><<<grid, 256, 0, s>>>(a);
  else linear_grad_kernel<Tile64, Tile128><<<grid, 256, 0, s>>>(a);
  hipError_t err = hipGetLastError();
  if (err == hipSuccess && a.n_dx && a.plan_dx.splits > 1) err = join(a.dx, a.plan_dx, a.out_dx, a.part_dx, s);
  if (err == hipSuccess && a.n_dw && a.plan_dw.splits > 1) err = join(a.dw, a.plan_dw, a.out_dw, a.part_dw, s);
  return err;
}

// Whether a call takes the kernels for few rows: by dot products always, on the matrix instruction
// where they are quicker than the tiles.  A workgroup a compute unit: a round takes 0.65 us and, for
// each 512 K, 0.2 to 0.7 as more units are busy (past 16 rows 0.65 to 0.9).  (us, these and tiles: 16 x
// 4096 x 4096 8.9, 12.1; 32 x 4096 x 4096 12.2, 12.6; 16 x 11008 x 4096 20.7, 32; 16 x 1024 x 8192 8.2,
// 12.7; 3 x 512 x 8192 7.2, 10.4; and the other way 4 x 50257 x 1600 44, 32; 32 x 50257 x 1600 65, 33;
// 32 x 2048 x 8192 15.2, 13.4.)
bool linear_takes_few(int64_t M, int64_t N, int64_t K) {
  if (M <= kLinearDotRows) return true;
  if (M > kLinearFewRows) return false;
  double tiles;
  best_plan(M, N, K, 64, 256, true, &tiles);
  const double groups = double(cdiv(N, 16)), busy = groups < 256 ? groups / 256 : 1;
  const double stage = M <= 16 ? 0.2 + 0.5 * busy : 0.65 + 0.25 * busy;
  return double(cdiv(int64_t(groups), 256)) * (0.65 + double(cdiv(K, 512)) * stage) + 2.5 < tiles;
}

hipError_t launch_linear_few(const LinearProduct& p, const LinearEpilogue& e, hipStream_t s) {
  if (p.M > kLinearDotRows) {
    const unsigned groups = (unsigned)((p.N + 15) / 16);
    if (p.M <= 16) linear_stream_kernel<1><<<groups, 256, 0, s>>>(p, e);
    else linear_stream_kernel<2><<<groups, 256, 0, s>>>(p, e);
    return hipGetLastError();
  }
  const int MT = p.M <= 1 ? 1 : 2;
  const int most = FEW_LDS / (2 * MT), k_stage = p.K < most ? p.K : most;
  const size_t lds = size_t(MT) * size_t(k_stage) * 2;
  const int per = 4 * FEW_R, groups = (p.N + per - 1) / per;
  const unsigned grid = (unsigned)(groups < 1024 ? groups : 1024);
  if (MT == 1) linear_few_kernel<1><<<grid, 256, lds, s>>>(p, e, k_stage);
  else linear_few_kernel<2><<<grid, 256, lds, s>>>(p, e, k_stage);
  return hipGetLastError();
}

// Shares of n: enough workgroups to fill the chip, few enough to join.
LinearPlan linear_few_dx_plan(int64_t M, int64_t N, int64_t K) {
  LinearPlan p = plan_of(64, 1, N);
  const int64_t blocks = cdiv(K, DX_COLS) * cdiv(M, DX_ROWS), want = cdiv(512, blocks), most = cdiv(N, DX_STAGE);
  int64_t splits = want < 96 ? want : 96;
  if (splits > most) splits = most;
  p.k_each = int(cdiv(N, splits));
  p.splits = int(cdiv(N, p.k_each));
  return p;
}

hipError_t launch_linear_few_dx(LinearFewDx a, const LinearPlan& plan, hipStream_t s) {
  a.each = plan.k_each;
  a.splits = plan.splits;
  a.lanes = 1;
  while (a.lanes < 64 && 8 * a.lanes < a.K) a.lanes *= 2;
  const dim3 grid((unsigned)cdiv(a.K, DX_COLS), (unsigned)a.splits, (unsigned)cdiv(a.M, DX_ROWS));
  if (a.dy_dtype == kF32) linear_few_dx_kernel<F32><<<grid, 256, 0, s>>>(a);
  else linear_few_dx_kernel<Bf16><<<grid, 256, 0, s>>>(a);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.splits == 1) return err;
  LinearProduct p{};
  p.M = a.M;
  p.N = a.K;
  LinearEpilogue e{};
  e.out = a.dx;
  e.out_dtype = kBf16;
  e.ldo = a.lddx;
  return join(p, plan, e, a.part, s);
}

int linear_slope_groups(int64_t M, int64_t N) {
  const int64_t cols = (N + SLOPE_COLS - 1) / SLOPE_COLS;
  int64_t g = 1024 / cols;
  const int64_t most = (M + 4 * SLOPE_ROWS - 1) / (4 * SLOPE_ROWS);
  if (g > most) g = most;
  return int(g < 1 ? 1 : g);
}

hipError_t launch_linear_slope(const LinearSlopeArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + SLOPE_COLS - 1) / SLOPE_COLS), (unsigned)a.groups);
  if (a.dy_dtype == kF32) {
    if (a.vec) linear_slope_kernel<F32, true><<<grid, 256, 0, s>>>(a);
    else linear_slope_kernel<F32, false><<<grid, 256, 0, s>>>(a);
  } else {
    if (a.vec) linear_slope_kernel<Bf16, true><<<grid, 256, 0, s>>>(a);
    else linear_slope_kernel<Bf16, false><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace flce
