// Layer norm for gfx950, forward and backward.
//
//   mean = sum_j x_j / H,  rstd = (sum_j (x_j - mean)^2 / H + eps)^-1/2,
//   xh = (x - mean) rstd,  y = weight xh + bias
//   g = weight dy,  dx = rstd (g - mean_j g - xh mean_j(g xh)),
//   dweight = sum_m dy xh,  dbias = sum_m dy
//
// All sums are in 32 bits.  The variance is that of the centred values, a second pass over
// registers that also sums the centred values themselves: their mean is what the first pass
// got wrong, and correcting both statistics by it makes an offset much larger than the
// spread cost no digits (a constant row is centred to exact zeros).  Both directions are
// bound by memory: every element is read once and written once.  A row lives in registers, 8
// consecutive elements a chunk: those of one wave or less up to H = 512 in the forward and 1024
// in the backward, of one workgroup up to 16384 and 8192.  Longer rows are read again from
// memory for every pass (three in the forward; in the backward one for the column sums and two
// for dx).
// The forward can write a microscaled 8-bit copy of x on the way (the quad of lanes that
// holds a block of 32 finds its scale), and the backward can read that copy in place of x.
//
// The backward's workgroups each walk many rows and keep the column sums of dweight and
// dbias in registers; each leaves one row of partial sums, and a second kernel adds those in
// a fixed order: no atomics, so results are bitwise repeatable.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "ops_internal.h"

namespace flce {

namespace {

// The sum over the LANES (16, 32 or 64) neighbouring lanes of a row, in every one of them.
template <int CTRL>
__device__ __forceinline__ float dpp_sum(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  v = dpp_sum<0xB1>(v);   // lane ^ 1
  v = dpp_sum<0x4E>(v);   // lane ^ 2
  v = dpp_sum<0x141>(v);  // the other quad of 8 lanes (half-row mirror)
  v = dpp_sum<0x140>(v);  // the other 8 lanes of 16 (row mirror)
  if constexpr (LANES > 16) v += __shfl_xor(v, 16);
  if constexpr (LANES > 32) v += __shfl_xor(v, 32);
  return v;
}

// Threads of a workgroup for rows of NT threads, and rows it holds: those of a wave or less
// need no barrier and share a workgroup of four waves.
constexpr int threads_of(int nt) { return nt <= 64 ? 256 : nt; }
constexpr int rows_of(int nt) { return threads_of(nt) / nt; }

// Sums of N <= 2 values over the NT threads that share a row (in every thread).  More than
// one wave meet in LDS; `buf` (2 x NT / 64 x 2 floats) alternates halves, so that one barrier
// a call is enough: a wave can only write a half again after the barrier of the call between,
// which every wave reaches after it has read that half.
template <int NT>
struct RowSum {
  float* buf;
  int turn = 0;
  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum<NT < 64 ? NT : 64>(v[i]);
    if constexpr (NT > 64) {
      constexpr int W = NT / 64;
      float* b = buf + turn * (2 * W);
      turn ^= 1;
      const int wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) b[wave * N + i] = v[i];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float s = b[i];
#pragma unroll
        for (int w = 1; w < W; ++w) s += b[w * N + i];
        v[i] = s;
      }
    }
  }
};

// 1 / sqrt(variance + eps) from the mean square about a value `off` away from the mean.
__device__ __forceinline__ float row_rstd(float square, float off, float eps) {
  const float var = fmaf(-off, off, square);
  return 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);  // NaN stays NaN
}

// Elements [col, col + 8) of a parameter vector (or `other` everywhere without one), 0 past
// the end.
template <bool VEC>
__device__ __forceinline__ void load_param(const void* p, int dtype, int col, int H, float other,
                                           float (&v)[8]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = col + i < H ? other : 0.f;
  } else if (dtype == kF32) {
    load8<F32, VEC>(static_cast<const float*>(p), col, H, v);
  } else {
    load8<Bf16, VEC>(static_cast<const uint16_t*>(p), col, H, v);
  }
}

// One block's share of a checkpoint row: 8 codes, and the scale byte from the quad's first
// lane.
template <int FMT>
__device__ __forceinline__ void save8(const float (&v)[8], int col, uint8_t* codes, uint8_t* scales) {
  const uint32_t byte = mx_scale_byte<FMT>(v);
  *reinterpret_cast<u32x2_t*>(codes + col) = mx_encode<FMT>(v, byte);
  if ((col & 31) == 0) scales[col >> 5] = (uint8_t)byte;
}

// Rows of H <= 8 NT CH elements, NT threads a row.
template <class TX, class TY, int NT, int CH, bool VEC>
__global__ __launch_bounds__(threads_of(NT)) void norm_fwd_kernel(NormFwdArgs p) {
  constexpr int ROWS = rows_of(NT);
  __shared__ float red[4 * ((NT + 63) / 64)];
  const int t = threadIdx.x % NT, H = p.H;
  RowSum<NT> sum{red};
  float w[CH][8], b[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    load_param<VEC>(p.weight, p.param_dtype, 8 * (t + NT * c), H, 1.f, w[c]);
    load_param<VEC>(p.bias, p.param_dtype, 8 * (t + NT * c), H, 0.f, b[c]);
  }
  const float rh = 1.f / (float)H;
  const long code_ld = mx_code_bytes(H, kMxFp8), scale_ld = mx_scale_bytes(H);
  // rows are uniform over the threads that meet at a barrier
  for (long row = (long)blockIdx.x * ROWS + threadIdx.x / NT; row < p.M; row += (long)gridDim.x * ROWS) {
    const typename TX::mem* x = static_cast<const typename TX::mem*>(p.x) + row * p.ldx;
    float v[CH][8];
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) load8<TX, VEC>(x, 8 * (t + NT * c), H, v[c]);
    if (p.fmt != kMxNone) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = 8 * (t + NT * c);
        // whole quads: the codes' rows end with a whole block
        if (col < code_ld) {
          if (p.fmt == kMxFp8)
            save8<kMxFp8>(v[c], col, p.codes + row * code_ld, p.scales + row * scale_ld);
          else
            save8<kMxInt8>(v[c], col, p.codes + row * code_ld, p.scales + row * scale_ld);
        }
      }
      for (long i = mx_blocks(H) + t; i < scale_ld; i += NT) p.scales[row * scale_ld + i] = 0;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += v[c][i];
    sum(s);
    const float first = s[0] / (float)H;
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = 8 * (t + NT * c) + (VEC ? 0 : i) < H ? v[c][i] - first : 0.f;
        v[c][i] = d;
        q[0] += d;
        q[1] = fmaf(d, d, q[1]);
      }
    sum(q);
    const float off = q[0] * rh, mean = first + off;
    const float rstd = row_rstd(q[1] * rh, off, p.eps);
    typename TY::mem* y = static_cast<typename TY::mem*>(p.y) + row * p.ldy;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = fmaf((v[c][i] - off) * rstd, w[c][i], b[c][i]);
      store8<TY, VEC>(y, 8 * (t + NT * c), H, o);
    }
    if (t == 0) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
  }
}

// The backward's view of the input: a matrix of T, or its 8-bit checkpoint.
struct Saved {};
template <class TX, bool VEC>
struct Input {
  Chunk8<TX, VEC> c;
  __device__ __forceinline__ void load(const NormBwdArgs& p, long row, int col) {
    c.load(static_cast<const typename TX::mem*>(p.x) + row * p.ldx, col, p.H);
  }
  __device__ __forceinline__ void value(const NormBwdArgs& p, int col, float (&o)[8]) const {
    c.value(col, p.H, o);
  }
};
template <bool VEC>
struct Input<Saved, VEC> {
  u32x2_t r;
  uint32_t byte;
  __device__ __forceinline__ void load(const NormBwdArgs& p, long row, int col) {
    const long code_ld = mx_code_bytes(p.H, kMxFp8), scale_ld = mx_scale_bytes(p.H);
    r = u32x2_t{0u, 0u};
    byte = 0u;
    if (col < code_ld) {
      r = *reinterpret_cast<const u32x2_t*>(p.codes + row * code_ld + col);
      byte = p.scales[row * scale_ld + (col >> 5)];
    }
  }
  __device__ __forceinline__ void value(const NormBwdArgs& p, int, float (&o)[8]) const {
    if (p.fmt == kMxFp8)
      mx_decode<kMxFp8>(r, byte, o);
    else
      mx_decode<kMxInt8>(r, byte, o);
  }
};

// Rows of H <= 8 NT CH elements; group g of the launch takes rows g, g + groups, ..., with
// the next row's loads in flight under the work on this one, and leaves the column sums of
// its rows.  Rows that share a workgroup join their sums in LDS first, in order.
template <class TX, class TY, class TD, int NT, int CH, bool VEC>
__global__ __launch_bounds__(threads_of(NT)) void norm_bwd_kernel(NormBwdArgs p) {
  constexpr int ROWS = rows_of(NT);
  __shared__ float red[4 * ((NT + 63) / 64)];
  __shared__ float join[ROWS > 1 ? 16 * NT * CH : 1];
  const int t = threadIdx.x % NT, slot = threadIdx.x / NT, H = p.H;
  RowSum<NT> sum{red};
  float w[CH][8], dw[CH][8], db[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    load_param<VEC>(p.weight, p.param_dtype, 8 * (t + NT * c), H, 1.f, w[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = db[c][i] = 0.f;
  }
  const float rh = 1.f / (float)H;
  struct Row {
    Input<TX, VEC> x[CH];
    Chunk8<TY, VEC> dy[CH];
    float mean, rstd;
    __device__ __forceinline__ void load(const NormBwdArgs& p, long row, int t) {
      const typename TY::mem* dyr = static_cast<const typename TY::mem*>(p.dy) + row * p.lddy;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        x[c].load(p, row, 8 * (t + NT * c));
        dy[c].load(dyr, 8 * (t + NT * c), p.H);
      }
      mean = p.mean[row];
      rstd = p.rstd[row];
    }
  } next;
  const long step = (long)gridDim.x * ROWS;
  long row = (long)blockIdx.x * ROWS + slot;
  if (row < p.M) next.load(p, row, t);
  for (; row < p.M; row += step) {
    const Row cur = next;
    if (row + step < p.M) next.load(p, row + step, t);
    const float mean = cur.mean, rstd = cur.rstd;
    float x[CH][8], g[CH][8];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      cur.x[c].value(p, 8 * (t + NT * c), x[c]);
      cur.dy[c].value(8 * (t + NT * c), H, g[c]);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // past the row g is 0, and so is its share of every sum
        const float xh = (x[c][i] - mean) * rstd;
        dw[c][i] = fmaf(g[c][i], xh, dw[c][i]);
        db[c][i] += g[c][i];
        g[c][i] *= w[c][i];
        x[c][i] = xh;
        s[0] += g[c][i];
        s[1] = fmaf(g[c][i], xh, s[1]);
      }
    sum(s);
    const float m0 = s[0] * rh, m1 = s[1] * rh;
    typename TD::mem* dx = static_cast<typename TD::mem*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = rstd * (g[c][i] - m0 - x[c][i] * m1);
      store8<TD, VEC>(dx, 8 * (t + NT * c), H, o);
    }
  }
  if constexpr (ROWS > 1) {
    // slot 0 adds the other slots' sums to its own, one slot after another
    float* jw = join + 16 * CH * t;
    for (int k = 1; k < ROWS; ++k) {
      if (slot == k) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            jw[16 * c + i] = dw[c][i];
            jw[16 * c + 8 + i] = db[c][i];
          }
      }
      __syncthreads();
      if (slot == 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dw[c][i] += jw[16 * c + i];
            db[c][i] += jw[16 * c + 8 + i];
          }
      }
      __syncthreads();
    }
    if (slot != 0) return;
  }
  float* pw = p.part + (long)blockIdx.x * H;
  float* pb = pw + (long)p.groups * H;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    store8<F32, VEC>(pw, 8 * (t + NT * c), H, dw[c]);
    store8<F32, VEC>(pb, 8 * (t + NT * c), H, db[c]);
  }
}

// Rows too long for a workgroup's registers: passes over memory (the row is in L2 after the
// first).  Thread t takes chunks t, t + 1024, ...
constexpr int WIDE = 1024;
template <class TX, class TY, bool VEC>
__global__ __launch_bounds__(WIDE) void norm_fwd_wide_kernel(NormFwdArgs p) {
  __shared__ float red[4 * (WIDE / 64)];
  RowSum<WIDE> sum{red};
  const int t = threadIdx.x, H = p.H;
  const float rh = 1.f / (float)H;
  const long code_ld = mx_code_bytes(H, kMxFp8), scale_ld = mx_scale_bytes(H);
  for (long row = blockIdx.x; row < p.M; row += gridDim.x) {
    const typename TX::mem* x = static_cast<const typename TX::mem*>(p.x) + row * p.ldx;
    float s[1] = {0.f};
    float v[8], w[8], b[8];
    for (int col = 8 * t; col < code_ld; col += 8 * WIDE) {
      load8<TX, VEC>(x, col, H, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += v[i];
      if (p.fmt == kMxFp8)
        save8<kMxFp8>(v, col, p.codes + row * code_ld, p.scales + row * scale_ld);
      else if (p.fmt == kMxInt8)
        save8<kMxInt8>(v, col, p.codes + row * code_ld, p.scales + row * scale_ld);
    }
    if (p.fmt != kMxNone)
      for (long i = mx_blocks(H) + t; i < scale_ld; i += WIDE) p.scales[row * scale_ld + i] = 0;
    sum(s);
    const float first = s[0] / (float)H;
    float q[2] = {0.f, 0.f};
    for (int col = 8 * t; col < H; col += 8 * WIDE) {
      load8<TX, VEC>(x, col, H, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = col + i < H ? v[i] - first : 0.f;
        q[0] += d;
        q[1] = fmaf(d, d, q[1]);
      }
    }
    sum(q);
    const float off = q[0] * rh, mean = first + off;
    const float rstd = row_rstd(q[1] * rh, off, p.eps);
    typename TY::mem* y = static_cast<typename TY::mem*>(p.y) + row * p.ldy;
    for (int col = 8 * t; col < H; col += 8 * WIDE) {
      load8<TX, VEC>(x, col, H, v);
      load_param<VEC>(p.weight, p.param_dtype, col, H, 1.f, w);
      load_param<VEC>(p.bias, p.param_dtype, col, H, 0.f, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf((v[i] - first - off) * rstd, w[i], b[i]);
      store8<TY, VEC>(y, col, H, v);
    }
    if (t == 0) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
  }
}

// The backward of such rows reads x and dy once for the column sums and once for dx (with the
// column sums in the workgroup's row of partial sums, read and written for every row, 3000 x
// 20000 bf16 took 253 us instead of 141).  Column sums: a thread's 8 columns over the rows of
// group blockIdx.y.
template <class TX, class TY, bool VEC>
__global__ __launch_bounds__(256) void norm_bwd_columns_kernel(NormBwdArgs p) {
  const int H = p.H, col = 8 * ((int)blockIdx.x * 256 + (int)threadIdx.x);
  if (col >= H) return;
  float dw[8], db[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.f;
#pragma unroll 4
  for (long row = blockIdx.y; row < p.M; row += p.groups) {
    Input<TX, VEC> in;
    Chunk8<TY, VEC> c;
    in.load(p, row, col);
    c.load(static_cast<const typename TY::mem*>(p.dy) + row * p.lddy, col, H);
    const float mean = p.mean[row], rstd = p.rstd[row];
    float x[8], dy[8];
    in.value(p, col, x);
    c.value(col, H, dy);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[i] = fmaf(dy[i], (x[i] - mean) * rstd, dw[i]);
      db[i] += dy[i];
    }
  }
  float* pw = p.part + (long)blockIdx.y * H;
  store8<F32, VEC>(pw, col, H, dw);
  store8<F32, VEC>(pw + (long)p.groups * H, col, H, db);
}

template <class TX, class TY, class TD, bool VEC>
__global__ __launch_bounds__(WIDE) void norm_bwd_wide_kernel(NormBwdArgs p) {
  __shared__ float red[4 * (WIDE / 64)];
  RowSum<WIDE> sum{red};
  const int t = threadIdx.x, H = p.H;
  const float rh = 1.f / (float)H;
  for (long row = blockIdx.x; row < p.M; row += gridDim.x) {
    const typename TY::mem* dy = static_cast<const typename TY::mem*>(p.dy) + row * p.lddy;
    typename TD::mem* dx = static_cast<typename TD::mem*>(p.dx) + row * p.lddx;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s[2] = {0.f, 0.f};
    float x[8], g[8], w[8];
    for (int col = 8 * t; col < H; col += 8 * WIDE) {
      Input<TX, VEC> in;
      in.load(p, row, col);
      in.value(p, col, x);
      load8<TY, VEC>(dy, col, H, g);
      load_param<VEC>(p.weight, p.param_dtype, col, H, 1.f, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // past the row g is 0, and so is its share of both sums
        g[i] *= w[i];
        s[0] += g[i];
        s[1] = fmaf(g[i], (x[i] - mean) * rstd, s[1]);
      }
    }
    sum(s);
    const float m0 = s[0] * rh, m1 = s[1] * rh;
    for (int col = 8 * t; col < H; col += 8 * WIDE) {
      Input<TX, VEC> in;
      in.load(p, row, col);
      in.value(p, col, x);
      load8<TY, VEC>(dy, col, H, g);
      load_param<VEC>(p.weight, p.param_dtype, col, H, 1.f, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = rstd * (g[i] * w[i] - m0 - (x[i] - mean) * rstd * m1);
      store8<TD, VEC>(dx, col, H, x);
    }
  }
}

// dweight and dbias: the sum of the groups' partial rows, in a fixed order.  A workgroup
// takes 32 columns (whole lines of the partial rows; of 16 columns, 2 to 3 us more at H = 8192);
// 32 slices of threads share the groups and meet in LDS.
constexpr int REDUCE_COLS = 32, REDUCE_SLICES = 32;
__global__ __launch_bounds__(REDUCE_COLS * REDUCE_SLICES) void norm_reduce_kernel(NormReduceArgs p) {
  __shared__ float part[REDUCE_SLICES][REDUCE_COLS];
  const int lane = threadIdx.x % REDUCE_COLS, slice = threadIdx.x / REDUCE_COLS;
  const int per = (p.H + REDUCE_COLS - 1) / REDUCE_COLS;
  const bool bias = (int)blockIdx.x >= per;
  void* out = bias ? p.dbias : p.dweight;
  const long col = (long)((int)blockIdx.x - (bias ? per : 0)) * REDUCE_COLS + lane;
  if (!out) return;  // uniform over the workgroup
  const float* src = p.part + (bias ? (long)p.groups * p.H : 0) + col;
  float s = 0.f;
  if (col < p.H) {
#pragma unroll 8
    for (int g = slice; g < p.groups; g += REDUCE_SLICES) s += src[(long)g * p.H];
  }
  part[slice][lane] = s;
  __syncthreads();
  // halves of the slices onto one another, in a fixed order
#pragma unroll
  for (int n = REDUCE_SLICES / 2; n > 0; n /= 2) {
    if (slice < n) part[slice][lane] += part[slice + n][lane];
    __syncthreads();
  }
  if (slice != 0 || col >= p.H) return;
  s = part[0][lane];
  if (p.param_dtype == kF32)
    static_cast<float*>(out)[col] = s;
  else
    static_cast<uint16_t*>(out)[col] = Bf16::from_f32(s);
}

constexpr int kComputeUnits = 256;

// A row takes as many threads as it has chunks where that is at most 1024: one chunk a
// thread keeps the registers few and the waves in flight many (32767 x 2048 bf16 forward:
// 49 us with 256 threads of one chunk a row, 78 us with a wave of four).  Past 4096 elements
// the forward gives a thread two (8192 x 8192: 59 us against 75 us with 1024 threads, whose
// barriers span 16 waves); the backward, with its column sums in registers, does not (88 us
// against 119 us before its loads ran ahead), but keeps rows of up to 1024 in a wave, without
// a barrier (65535 x 1024: 79 us against 85 us).  Workgroups stay and walk the rows, so each
// reads the parameters once.
template <class TX, class TY, bool VEC>
void fwd_rows(const NormFwdArgs& a, hipStream_t s) {
  auto grid = [&](int rows_per_group, int groups_per_unit) {
    const long need = (a.M + rows_per_group - 1) / rows_per_group;
    const long most = (long)kComputeUnits * groups_per_unit;
    return (unsigned)(need < most ? need : most);
  };
  if (a.H <= 128)
    norm_fwd_kernel<TX, TY, 16, 1, VEC><<<grid(16, 16), 256, 0, s>>>(a);
  else if (a.H <= 256)
    norm_fwd_kernel<TX, TY, 32, 1, VEC><<<grid(8, 16), 256, 0, s>>>(a);
  else if (a.H <= 512)
    norm_fwd_kernel<TX, TY, 64, 1, VEC><<<grid(4, 16), 256, 0, s>>>(a);
  else if (a.H <= 1024)
    norm_fwd_kernel<TX, TY, 128, 1, VEC><<<grid(1, 32), 128, 0, s>>>(a);
  else if (a.H <= 2048)
    norm_fwd_kernel<TX, TY, 256, 1, VEC><<<grid(1, 16), 256, 0, s>>>(a);
  else if (a.H <= 4096)
    norm_fwd_kernel<TX, TY, 512, 1, VEC><<<grid(1, 8), 512, 0, s>>>(a);
  else if (a.H <= 8192)
    norm_fwd_kernel<TX, TY, 512, 2, VEC><<<grid(1, 4), 512, 0, s>>>(a);
  else if (a.H <= 16384)
    norm_fwd_kernel<TX, TY, 1024, 2, VEC><<<grid(1, 2), 1024, 0, s>>>(a);
  else
    norm_fwd_wide_kernel<TX, TY, VEC><<<grid(1, 2), WIDE, 0, s>>>(a);
}

template <class TX, class TY, class TD, bool VEC>
void bwd_rows(const NormBwdArgs& a, hipStream_t s) {
  const unsigned g = (unsigned)a.groups;
  if (a.H <= 128)
    norm_bwd_kernel<TX, TY, TD, 16, 1, VEC><<<g, 256, 0, s>>>(a);
  else if (a.H <= 256)
    norm_bwd_kernel<TX, TY, TD, 32, 1, VEC><<<g, 256, 0, s>>>(a);
  else if (a.H <= 512)
    norm_bwd_kernel<TX, TY, TD, 64, 1, VEC><<<g, 256, 0, s>>>(a);
  else if (a.H <= 1024)
    norm_bwd_kernel<TX, TY, TD, 64, 2, VEC><<<g, 256, 0, s>>>(a);
  else if (a.H <= 2048)
    norm_bwd_kernel<TX, TY, TD, 256, 1, VEC><<<g, 256, 0, s>>>(a);
  else if (a.H <= 4096)
    norm_bwd_kernel<TX, TY, TD, 512, 1, VEC><<<g, 512, 0, s>>>(a);
  else if (a.H <= 8192)
    norm_bwd_kernel<TX, TY, TD, 1024, 1, VEC><<<g, 1024, 0, s>>>(a);
  else {
    // (the columns first: dx may overwrite x or dy)
    if (a.params)
      norm_bwd_columns_kernel<TX, TY, VEC><<<dim3((a.H + 2047) / 2048, g), 256, 0, s>>>(a);
    const long most = 2 * kComputeUnits;
    norm_bwd_wide_kernel<TX, TY, TD, VEC><<<(unsigned)(a.M < most ? a.M : most), WIDE, 0, s>>>(a);
  }
}

template <class TX, class TY, class TD>
void bwd_vec(const NormBwdArgs& a, bool vec, hipStream_t s) {
  if (vec) bwd_rows<TX, TY, TD, true>(a, s);
  else bwd_rows<TX, TY, TD, false>(a, s);
}
template <class TX, class TY>
void fwd_vec(const NormFwdArgs& a, bool vec, hipStream_t s) {
  if (vec) fwd_rows<TX, TY, true>(a, s);
  else fwd_rows<TX, TY, false>(a, s);
}

}  // namespace

// Workgroups of the backward's row kernel.  Each leaves two rows of partial sums, and the next
// row's loads in flight keep memory busy with few of them (us with 1, 2, 3, 4 a compute unit:
// 65535 x 1024 77, 78, -, 88; 32767 x 2048 110, 77, 79, 84, and from the checkpoint 111, 74,
// 67, 70; 16384 x 4096 77, 82, 91; 8192 x 8192 84, 91).  Past one a unit each has 16 turns.
int norm_bwd_groups(long M, int H) {
  const long rows = H <= 128 ? 16 : H <= 256 ? 8 : H <= 1024 ? 4 : 1;
  const long most = kComputeUnits * (H <= 512 ? 2 : H <= 1024 ? 1 : H <= 2048 ? 3 : 1);
  const long need = (M + rows - 1) / rows;
  const long shared = need / 16 > kComputeUnits ? need / 16 : kComputeUnits;
  const long g = need < shared ? need : shared;
  return (int)(g < most ? g : most);
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, int x_dtype, int y_dtype, bool vec, hipStream_t s) {
  if (x_dtype == kBf16) fwd_vec<Bf16, Bf16>(a, vec, s);
  else if (y_dtype == kBf16) fwd_vec<F32, Bf16>(a, vec, s);
  else fwd_vec<F32, F32>(a, vec, s);
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, int x_dtype, int dy_dtype, int dx_dtype, bool vec,
                           hipStream_t s) {
  if (!a.x) {
    if (dx_dtype == kBf16) bwd_vec<Saved, Bf16, Bf16>(a, vec, s);
    else if (dy_dtype == kBf16) bwd_vec<Saved, Bf16, F32>(a, vec, s);
    else bwd_vec<Saved, F32, F32>(a, vec, s);
  } else if (x_dtype == kBf16) {
    bwd_vec<Bf16, Bf16, Bf16>(a, vec, s);
  } else if (dy_dtype == kBf16) {
    bwd_vec<F32, Bf16, F32>(a, vec, s);
  } else {
    bwd_vec<F32, F32, F32>(a, vec, s);
  }
  return hipGetLastError();
}

hipError_t launch_norm_reduce(const NormReduceArgs& a, hipStream_t s) {
  const unsigned per = (unsigned)((a.H + REDUCE_COLS - 1) / REDUCE_COLS);
  norm_reduce_kernel<<<2 * per, REDUCE_COLS * REDUCE_SLICES, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace flce
