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
// second kernel.  A decoding step (up to 8 rows) has a kernel of its own that streams W.
#include <hip/hip_runtime.h>
#include <stdint.h>

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
// error (6e-8; 4e-7 with fp32 arithmetic).  The library's erff takes twice as long.
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

__device__ __forceinline__ float activate(float x, int act) {
  switch (act) {
    case kActRelu: return x < 0.f ? 0.f : x;
    case kActGelu: {
      float ex;
      return x * normal_cdf(x, ex);
    }
    // (1 + tanh u) / 2 is the logistic function of 2 u
    case kActGeluTanh: return x * logistic(TANH_SCALE * x * fmaf(TANH_CUBE * x, x, 1.f));
    case kActSilu: return x * logistic(x);
    default: return x;
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
// (the branch is the same for every lane)
__device__ __forceinline__ void activate8(float (&v)[8], int act) {
  if (act == kActNone) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = activate(v[i], act);
}

// ---------------------------------------------------------------------------
// The epilogue of 8 consecutive columns of a row.
template <bool VEC>
__device__ __forceinline__ void load_any(const void* p, int dtype, long at, int col, int N, float (&v)[8]) {
  if (dtype == kF32) load8<F32, VEC>(static_cast<const float*>(p) + at, col, N, v);
  else load8<Bf16, VEC>(static_cast<const uint16_t*>(p) + at, col, N, v);
}
template <bool VEC>
__device__ __forceinline__ void finish8(const LinearEpilogue& e, long m, int col, int N, float (&v)[8]) {
  if (e.bias) {
    float b[8];
    load_any<VEC>(e.bias, e.bias_dtype, 0, col, N, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  if (e.pre) store8<Bf16, VEC>(e.pre + m * e.ldp, col, N, v);
  activate8(v, e.act);
  if (e.residual) {
    float r[8];
    load_any<VEC>(e.residual, e.residual_dtype, m * e.ldr, col, N, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  if (e.out_dtype == kF32) store8<F32, VEC>(static_cast<float*>(e.out) + m * e.ldo, col, N, v);
  else store8<Bf16, VEC>(static_cast<uint16_t*>(e.out) + m * e.ldo, col, N, v);
}

// A wave's accumulators (WM x WN of the tile at (m0, n0)) to the epilogue, 64 rows at a time
// through its own slice of LDS: row r, column c at float r WN + (c ^ 32 ((r >> 2) & 1)), so that
// the two half-waves of a write (rows r and r + 4) meet different banks where rows are 64 columns
// or more.  With `part` the fp32 values go there as they are.
template <class S, bool VEC>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[S::MB][S::NB], char* smem, const LinearEpilogue& e,
                                           float* part, long ldpart, int M, int N, int m0, int n0) {
  constexpr int WN = S::WN, ROWS = 64, BLOCKS = ROWS / 32, COLS8 = WN / 8, PER = 64 / COLS8;
  static_assert(S::MB % BLOCKS == 0 && S::NWAVES * ROWS * WN * 4 <= S::PIPE_BYTES, "slices");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* sl = reinterpret_cast<float*>(smem) + wave * ROWS * WN;
  const int lc = lane & 31, hi = lane >> 5, sw = WN >= 64 ? hi << 5 : 0;
  const int row0 = m0 + (wave / S::WAVES_N) * S::WM, col0 = n0 + (wave % S::WAVES_N) * WN;
  const int col = col0 + 8 * (lane % COLS8);
#pragma unroll
  for (int s = 0; s < S::MB / BLOCKS; ++s) {
#pragma unroll
    for (int mi = 0; mi < BLOCKS; ++mi)
#pragma unroll
      for (int nb = 0; nb < S::NB; ++nb)
#pragma unroll
        for (int q = 0; q < 16; ++q)
          sl[(32 * mi + acc_row(lane, q)) * WN + ((32 * nb + lc) ^ sw)] = acc_read(acc[BLOCKS * s + mi][nb][q]);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    // (not unrolled further: the unrolled block would be too long for the loop over s to be)
#pragma unroll 2
    for (int it = 0; it < ROWS / PER; ++it) {
      const int r = PER * it + lane / COLS8, m = row0 + ROWS * s + r;
      const int c = (8 * (lane % COLS8)) ^ (WN >= 64 ? ((r >> 2) & 1) << 5 : 0);
      const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(sl + r * WN + c);
      const f32x4_t up = *reinterpret_cast<const f32x4_t*>(sl + r * WN + c + 4);
      if (m < M && col < N) {
        if (part) {
          float* to = part + (long)m * ldpart + col;
          *reinterpret_cast<f32x4_t*>(to) = lo;
          *reinterpret_cast<f32x4_t*>(to + 4) = up;
        } else {
          float v[8] = {lo[0], lo[1], lo[2], lo[3], up[0], up[1], up[2], up[3]};
          finish8<VEC>(e, m, col, N, v);
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// A tile of TM x TN over a share of K.  Workgroups of one XCD take neighbouring tiles of the same
// share (groups of 8 tile rows).
template <class S, bool A_KC, bool B_KC, bool VEC>
__global__ __launch_bounds__(S::NTHREADS, S::WAVES_PER_EU) void linear_tile_kernel(LinearProduct p,
                                                                                  LinearEpilogue e, float* part,
                                                                                  long ldpart, int n_mt, int n_nt,
                                                                                  int splits, int k_each) {
  __shared__ __attribute__((aligned(1024))) char smem[S::PIPE_BYTES];
  const int tiles = n_mt * n_nt, per = (int)gridDim.x >> 3;
  int L = blockIdx.x;
  if (L < (per << 3)) L = (L & 7) * per + (L >> 3);
  const int split = L / tiles;
  int mt, nt;
  group_coords(L - split * tiles, n_mt, n_nt, 8, mt, nt);
  const int m0 = mt * S::TM, n0 = nt * S::TN;
  const int k0 = split * k_each, k1 = min(p.K, k0 + k_each);
  const TileSrc A{A_KC ? p.a + (long)m0 * p.lda + k0 : p.a + (long)k0 * p.lda + m0, p.lda, p.M - m0,
                  min(p.kvalid_a, k1) - k0, 0};
  const TileSrc B{B_KC ? p.b + (long)n0 * p.ldb + k0 : p.b + (long)k0 * p.ldb + n0, p.ldb, p.N - n0,
                  min(p.kvalid_b, k1) - k0, 0};
  f32x16 acc[S::MB][S::NB];
  mainloop<S, A_KC, B_KC>(acc, smem, A, B, k1 - k0);
  float* mine = splits > 1 ? part + (long)split * p.M * ldpart : nullptr;
  store_tile<S, VEC>(acc, smem, e, mine, ldpart, p.M, p.N, m0, n0);
}

// The partial products of a split K, added in order, and the epilogue: 8 columns a thread.
template <bool VEC>
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
    finish8<VEC>(e, m, col, N, v);
  }
}

// ---------------------------------------------------------------------------
// Up to MT <= 8 rows of X: W is read once, and bounds the call.  A wave takes R rows of W, its
// lanes 8 consecutive K each (1 KiB of a row at once), two steps of loads ahead; X lies in LDS,
// at most 64 KiB of it at a time, and is read from there once for the R rows.  Products of a
// pair of bf16 go through v_dot2: two multiplications and no unpacking (with unpacking and
// fp32 fused multiply-adds 8 rows of X would take more time than the loads of W).
constexpr int FEW_R = 4, FEW_LDS = 64 * 1024;
typedef __bf16 bf16x2_v __attribute__((ext_vector_type(2)));

template <int MT>
__global__ __launch_bounds__(256) void linear_few_kernel(LinearProduct p, LinearEpilogue e, int k_stage) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  constexpr int R = FEW_R, NVAL = R * MT;
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
      if (!staged) {
        __syncthreads();
        for (int i = threadIdx.x; i < MT * (len / 8); i += 256) {
          const int m = i / (len / 8), c = i - m * (len / 8);
          xs[m * ld8 + c] = m < p.M ? *reinterpret_cast<const u32x4_t*>(p.a + m * p.lda + ks + 8 * c) : zero;
        }
        __syncthreads();
        staged = k_stage >= p.K;
      }
      const uint16_t* w[R];
#pragma unroll
      for (int r = 0; r < R; ++r) w[r] = p.b + (long)min(n0 + r, p.N - 1) * p.ldb + ks;
      u32x4_t wv[2][R];
      auto load = [&](int b, int k) {
#pragma unroll
        for (int r = 0; r < R; ++r)
          wv[b][r] = k < len ? __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(w[r] + k)) : zero;
      };
      auto use = [&](int b, int k) {
        const int c = min(k, len - 8) / 8;  // (past the end W is zero, and X a number or not as it was)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const u32x4_t x = k < len ? xs[m * ld8 + c] : zero;
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // (values of their own: a cast of a vector's element takes the vector's first)
              const uint32_t wi = wv[b][r][i], xi = x[i];
              acc[r * MT + m] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_v, wi),
                                                                __builtin_bit_cast(bf16x2_v, xi),
                                                                acc[r * MT + m], false);
            }
        }
      };
      load(0, 8 * lane);
      load(1, 8 * lane + 512);
      for (int k = 0; k < len; k += 1024) {
        use(0, k + 8 * lane);
        load(0, k + 1024 + 8 * lane);
        use(1, k + 512 + 8 * lane);
        load(1, k + 1536 + 8 * lane);
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
    if ((lane & (64 / NVAL - 1)) == 0 && m < p.M && n < p.N) {
      if (e.bias)
        v += e.bias_dtype == kF32 ? static_cast<const float*>(e.bias)[n]
                                  : Bf16::to_f32(static_cast<const uint16_t*>(e.bias)[n]);
      if (e.pre) e.pre[m * e.ldp + n] = Bf16::from_f32(v);
      v = activate(v, e.act);
      if (e.residual)
        v += e.residual_dtype == kF32 ? static_cast<const float*>(e.residual)[m * e.ldr + n]
                                      : Bf16::to_f32(static_cast<const uint16_t*>(e.residual)[m * e.ldr + n]);
      if (e.out_dtype == kF32) static_cast<float*>(e.out)[m * e.ldo + n] = v;
      else static_cast<uint16_t*>(e.out)[m * e.ldo + n] = Bf16::from_f32(v);
    }
  }
}

// ---------------------------------------------------------------------------
// dpre = dy act'(pre), 8 columns a lane and 512 a workgroup, whose four waves walk the rows of
// its group; the column sums stay in registers and meet in LDS.
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

// The groups' column sums added in order: 32 columns a workgroup, 8 shares of the groups.
__global__ __launch_bounds__(256) void linear_bias_sum_kernel(const float* part, int groups, int N, void* dbias,
                                                              int dtype) {
  __shared__ float red[8][32];
  const int c = threadIdx.x & 31, sl = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  float s = 0.f;
  if (col < N)
    for (int g = sl; g < groups; g += 8) s += part[(long)g * N + col];
  red[sl][c] = s;
  __syncthreads();
  if (sl == 0 && col < N) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += red[k][c];
    if (dtype == kF32) static_cast<float*>(dbias)[col] = s;
    else static_cast<uint16_t*>(dbias)[col] = Bf16::from_f32(s);
  }
}

// ---------------------------------------------------------------------------
using Tile128 = Shape<128, 128, 64, 2, 2>;
using Tile64 = Shape<64, 128, 64, 2, 2, 1, 4>;

template <class S, bool A_KC, bool B_KC>
void run_tiles(const LinearProduct& p, const LinearPlan& plan, const LinearEpilogue& e, float* part, hipStream_t s) {
  const int n_mt = (p.M + S::TM - 1) / S::TM, n_nt = (p.N + S::TN - 1) / S::TN;
  const unsigned grid = (unsigned)n_mt * (unsigned)n_nt * (unsigned)plan.splits;
  const long ldpart = linear_part_ld(p.N);
  if (e.vec)
    linear_tile_kernel<S, A_KC, B_KC, true><<<grid, S::NTHREADS, 0, s>>>(p, e, part, ldpart, n_mt, n_nt, plan.splits,
                                                                         plan.k_each);
  else
    linear_tile_kernel<S, A_KC, B_KC, false><<<grid, S::NTHREADS, 0, s>>>(p, e, part, ldpart, n_mt, n_nt,
                                                                          plan.splits, plan.k_each);
}
template <bool A_KC, bool B_KC>
void run_plan(const LinearProduct& p, const LinearPlan& plan, const LinearEpilogue& e, float* part, hipStream_t s) {
  if (plan.tile_m == 256) {
    run_tiles<BigShape, A_KC, B_KC>(p, plan, e, part, s);
  } else if (plan.tile_m == 128) {
    run_tiles<Tile128, A_KC, B_KC>(p, plan, e, part, s);
  } else if constexpr (A_KC) {
    run_tiles<Tile64, A_KC, B_KC>(p, plan, e, part, s);
  }
}

}  // namespace

LinearPlan linear_plan(int64_t M, int64_t N, int64_t K, bool a_kc, bool b_kc) {
  (void)b_kc;
  auto cdiv = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  LinearPlan p{};
  const int64_t big = cdiv(M, 256) * cdiv(N, 256);
  if (big >= 192) p.tile_m = p.tile_n = 256;
  else if (M <= 64 && a_kc) p.tile_m = 64, p.tile_n = 128;
  else p.tile_m = p.tile_n = 128;
  const int64_t tiles = cdiv(M, p.tile_m) * cdiv(N, p.tile_n);
  int64_t splits = 1;
  if (p.tile_m < 256 && tiles > 0) {
    splits = 512 / tiles;
    if (splits > K / 512) splits = K / 512;
    if (splits < 1) splits = 1;
  }
  p.k_each = int(cdiv(cdiv(K > 0 ? K : 1, splits), 64) * 64);
  p.splits = int(cdiv(K > 0 ? K : 1, p.k_each));
  return p;
}

hipError_t launch_linear_product(const LinearProduct& p, const LinearPlan& plan, const LinearEpilogue& e, float* part,
                                 hipStream_t s) {
  if (p.a_kc && p.b_kc) run_plan<true, true>(p, plan, e, part, s);
  else if (p.a_kc) run_plan<true, false>(p, plan, e, part, s);
  else run_plan<false, false>(p, plan, e, part, s);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || plan.splits == 1) return err;
  const long total = (long)p.M * ((p.N + 7) / 8), need = (total + 255) / 256;
  const unsigned grid = (unsigned)(need < 4096 ? need : 4096);
  const long ldpart = linear_part_ld(p.N);
  if (e.vec) linear_join_kernel<true><<<grid, 256, 0, s>>>(e, part, ldpart, plan.splits, p.M, p.N);
  else linear_join_kernel<false><<<grid, 256, 0, s>>>(e, part, ldpart, plan.splits, p.M, p.N);
  return hipGetLastError();
}

hipError_t launch_linear_few(const LinearProduct& p, const LinearEpilogue& e, hipStream_t s) {
  const int MT = p.M <= 1 ? 1 : p.M <= 2 ? 2 : p.M <= 4 ? 4 : 8;
  const int most = FEW_LDS / (2 * MT), k_stage = p.K < most ? p.K : most;
  const size_t lds = size_t(MT) * size_t(k_stage) * 2;
  const int groups = (p.N + 4 * FEW_R - 1) / (4 * FEW_R);
  const unsigned grid = (unsigned)(groups < 1024 ? groups : 1024);
  if (MT == 1) linear_few_kernel<1><<<grid, 256, lds, s>>>(p, e, k_stage);
  else if (MT == 2) linear_few_kernel<2><<<grid, 256, lds, s>>>(p, e, k_stage);
  else if (MT == 4) linear_few_kernel<4><<<grid, 256, lds, s>>>(p, e, k_stage);
  else linear_few_kernel<8><<<grid, 256, lds, s>>>(p, e, k_stage);
  return hipGetLastError();
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

hipError_t launch_linear_bias_sum(const float* part, int groups, int N, void* dbias, int dtype, hipStream_t s) {
  linear_bias_sum_kernel<<<(unsigned)((N + 31) / 32), 256, 0, s>>>(part, groups, N, dbias, dtype);
  return hipGetLastError();
}

}  // namespace flce
