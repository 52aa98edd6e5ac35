// The head with 4-bit weights (gfx950): logits, or log-prob partials, of
//
//   z[m, v] = scale * sum_k X[m, k] W[v, k],  X and W in MXFP4
//
// on the scaled matrix instruction v_mfma_scale_f32_32x32x64_f8f6f4, which takes 32 e2m1
// codes of a row and their block's scale byte per lane (lane l: row l % 32, one block of the
// two that a call covers) and accumulates in fp32.  Products of codes are exact and the
// accumulators stay in fp32; nothing is rounded before the output.
//
// The contraction's order is free as long as both operands agree, so the blocks are dealt
// out to suit the loads: of the 8 blocks in 256 K (128 bytes of codes, one step), the lower
// half-wave takes blocks 0-3 and the upper 4-7, one each per instruction.  A lane's four
// scale bytes of a step are then one aligned dword, and the instruction picks byte kk.
//
//   mx_stream   few tokens: W streams from memory once, straight into registers, and bounds
//               the kernel; 8 waves of 32 vocabulary rows a workgroup.
//   mx_tile     many tokens: 256 x 256 tiles through LDS, bound by the matrix pipe.  A code
//               tile has the bytes of a bf16 tile of a quarter of the K, and an instruction
//               the cycles of a bf16 one, so the direct-to-LDS pipeline is that of the bf16
//               kernels, with the scales as a third, small stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "ops_internal.h"
#include "tile_device.h"

namespace flce {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kE2m1 = 4;  // the instruction's format code of e2m1

// Codes of one lane for one instruction, and D += A B^T of 32 rows each over 64 K with scale
// byte kk of sa and sb.
template <int kk>
__device__ __forceinline__ f32x16 mx_mfma(u32x4 a, u32x4 b, f32x16 c, int sa, int sb) {
  const i32x8 a8 = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8 b8 = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, kE2m1, kE2m1, kk, sa, kk, sb);
}

// ---------------------------------------------------------------------------
// Few tokens.
constexpr int STREAM_WAVES = 8, STREAM_ROWS = 32 * STREAM_WAVES;  // vocabulary rows a workgroup
static_assert(STREAM_ROWS == kFwdTileN, "partials of whole vocabulary tiles");

// One lane's share of a step: its four blocks of a row and their scale bytes.
struct StreamFrag {
  u32x4 c[4];
  uint32_t s;
};

// A lane's row of an operand: codes from block 4 (lane / 32), scales likewise.
struct StreamRow {
  const uint8_t* codes;
  const uint8_t* scales;
  int blocks;  // blocks of the row from this lane's first on (may be <= 0)
  __device__ __forceinline__ void init(const MxOperand& op, long row, int H, int half) {
    codes = op.codes + row * mx_code_bytes(H, kMxFp4) + 64 * half;
    scales = op.scales + row * mx_scale_bytes(H) + 4 * half;
    blocks = (int)mx_blocks(H) - 4 * half;
  }
  // step st; TAIL: blocks past the row's end read as zero codes
  template <bool TAIL>
  __device__ __forceinline__ void load(int st, StreamFrag& f) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!TAIL || 8 * st + j < blocks)
        f.c[j] = *reinterpret_cast<const u32x4*>(codes + 128l * st + 16 * j);
      else
        f.c[j] = u32x4{0u, 0u, 0u, 0u};
    }
    f.s = *reinterpret_cast<const uint32_t*>(scales + 8l * st);
  }
};

template <int TB>
struct StreamShape {
  static constexpr int MB = 1, NB = TB;
};

// acc[0][tb]: wave's 32 vocabulary rows x token block tb, as (A = W, B = X) for the log-probs
// (a lane then holds 16 vocabulary rows of one token) and as (A = X, B = W) for the logits (a
// lane holds one vocabulary column, so a store covers 128 contiguous bytes of a row).
template <int TB, bool LOGITS, int kk>
__device__ __forceinline__ void stream_mfma(f32x16 (&acc)[1][TB], const StreamFrag& w,
                                            const StreamFrag (&x)[TB]) {
#pragma unroll
  for (int tb = 0; tb < TB; ++tb)
    acc[0][tb] = LOGITS ? mx_mfma<kk>(x[tb].c[kk], w.c[kk], acc[0][tb], (int)x[tb].s, (int)w.s)
                        : mx_mfma<kk>(w.c[kk], x[tb].c[kk], acc[0][tb], (int)w.s, (int)x[tb].s);
}

template <int TB, bool LOGITS>
__device__ __forceinline__ void stream_step(f32x16 (&acc)[1][TB], const StreamFrag& w,
                                            const StreamFrag (&x)[TB]) {
  stream_mfma<TB, LOGITS, 0>(acc, w, x);
  stream_mfma<TB, LOGITS, 1>(acc, w, x);
  stream_mfma<TB, LOGITS, 2>(acc, w, x);
  stream_mfma<TB, LOGITS, 3>(acc, w, x);
}

// The products of 32 vocabulary rows from v0 and 32 TB tokens from m0.  Rows past the end
// repeat the last one; what they give is not used.
template <int TB, bool LOGITS>
__device__ __forceinline__ void stream_product(f32x16 (&acc)[1][TB], const MxOperand& xo,
                                               const MxOperand& wo, int M, int H, int V, int m0,
                                               int v0, int lane) {
  const int half = lane >> 5, r = lane & 31;
  StreamRow wr, xr[TB];
  wr.init(wo, min(v0 + r, V - 1), H, half);
#pragma unroll
  for (int tb = 0; tb < TB; ++tb) {
    xr[tb].init(xo, min(m0 + 32 * tb + r, M - 1), H, half);
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[0][tb][e] = 0.f;
  }
  const int nblk = (int)mx_blocks(H), full = nblk / 8, steps = (nblk + 7) / 8;
  StreamFrag w, x[TB];
  for (int st = 0; st < full; ++st) {
    wr.template load<false>(st, w);
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) xr[tb].template load<false>(st, x[tb]);
    stream_step<TB, LOGITS>(acc, w, x);
  }
  if (full < steps) {
    wr.template load<true>(full, w);
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) xr[tb].template load<true>(full, x[tb]);
    stream_step<TB, LOGITS>(acc, w, x);
  }
}

template <class T, int TB>
__global__ __launch_bounds__(64 * STREAM_WAVES) void mx_stream_logits_kernel(MxLogitsArgs p) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int vt = (int)(blockIdx.x % (unsigned)p.n_vt), mt = (int)(blockIdx.x / (unsigned)p.n_vt);
  const int m0 = mt * 32 * TB, v0 = vt * STREAM_ROWS + 32 * wave;
  if (v0 >= p.V) return;
  f32x16 acc[1][TB];
  stream_product<TB, true>(acc, p.x, p.w, p.M, p.H, p.V, m0, v0, lane);
  const int v = v0 + (lane & 31);
  if (v >= p.V) return;
  typename T::mem* out = static_cast<typename T::mem*>(p.out) + v;
#pragma unroll
  for (int tb = 0; tb < TB; ++tb)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int m = m0 + 32 * tb + acc_row(lane, e);
      if (m < p.M) out[(long)m * p.ldo] = T::from_f32(p.scale * acc[0][tb][e]);
    }
}

// Partials of one 256-entry vocabulary tile: maximum, then the shifted sums, each over the
// lane's 16 rows, the two half-waves and the 8 waves.
template <int TB, bool ENT>
__global__ __launch_bounds__(64 * STREAM_WAVES) void mx_stream_fwd_kernel(MxFwdArgs a) {
  using S = StreamShape<TB>;
  const FwdTileArgs& p = a.f;
  constexpr int TT = 32 * TB;
  __shared__ float red[STREAM_WAVES][TT];
  __shared__ float comb[2][STREAM_WAVES][TT];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int vt = (int)(blockIdx.x % (unsigned)p.n_vt), mt = (int)(blockIdx.x / (unsigned)p.n_vt);
  const int m0 = mt * TT, v0 = vt * STREAM_ROWS + 32 * wave;
  const int lc = lane & 31;
  f32x16 acc[1][TB];
  if (v0 < p.V)  // wave-uniform; the other waves of the tile only bring neutral partials
    stream_product<TB, false>(acc, a.x, a.w, p.M, p.H, p.V, m0, v0, lane);
  else
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[0][tb][e] = 0.f;
  const float c1 = p.scale * LOG2E, ac1 = fabsf(c1);
  const int vrows = p.V - v0;
  {
    float mx[TB];
    if (c1 >= 0.f) lane_col_max<false, true, S>(acc, lane, vrows, mx);
    else lane_col_max<true, true, S>(acc, lane, vrows, mx);
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
      const float m = halves_reduce(mx[tb], mx[tb], [](float x, float y) { return max_raw(x, y); });
      if (lane < 32) red[wave][32 * tb + lc] = m;
    }
  }
  __syncthreads();
  float nm2[TB], sv[TB], uv[TB];
#pragma unroll
  for (int tb = 0; tb < TB; ++tb) {
    float m = red[0][32 * tb + lc];
#pragma unroll
    for (int k = 1; k < STREAM_WAVES; ++k) m = fmaxf(m, red[k][32 * tb + lc]);
    nm2[tb] = -ac1 * m;
  }
  lane_col_sums<ENT, true, S>(acc, lane, vrows, c1, nm2, sv, uv);
#pragma unroll
  for (int tb = 0; tb < TB; ++tb) {
    const float s = halves_reduce(sv[tb], sv[tb], [](float x, float y) { return x + y; });
    const float u = halves_reduce(uv[tb], uv[tb], [](float x, float y) { return x + y; });
    if (lane < 32) {
      comb[0][wave][32 * tb + lc] = s;
      comb[1][wave][32 * tb + lc] = u;
    }
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t < TT && m0 + t < p.M) {
    float m = red[0][t], s = comb[0][0][t], u = comb[1][0][t];
#pragma unroll
    for (int k = 1; k < STREAM_WAVES; ++k) {
      m = fmaxf(m, red[k][t]);
      s += comb[0][k][t];
      u += comb[1][k][t];
    }
    const long off = (long)vt * p.Mpad + m0 + t;
    p.part_m[off] = ac1 * m * LN2;
    p.part_s[off] = s;
    if constexpr (ENT) p.part_u[off] = u * LN2;
  }
}

// Target logit of every row whose target W holds, one wave a row: lane i takes blocks i,
// i + 64, ...; a block's sum of code products is exact, its two scales multiply it once.
constexpr int TL_ROWS = 4;
__global__ __launch_bounds__(64 * TL_ROWS) void mx_target_logit_kernel(MxFwdArgs a) {
  const FwdTileArgs& p = a.f;
  // zero the tile kernel's queue counters: that kernel is launched after this one
  if (blockIdx.x == 0 && threadIdx.x < 8 && p.tq.ctr)
    __hip_atomic_store(&p.tq.ctr[threadIdx.x], 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const int lane = threadIdx.x & 63;
  const long row = (long)blockIdx.x * TL_ROWS + (threadIdx.x >> 6);
  if (row >= p.M) return;
  const int64_t t = p.targets[row];
  if (t == p.ignore_index || t < 0 || t >= p.V) return;
  const long code_ld = mx_code_bytes(p.H, kMxFp4), scale_ld = mx_scale_bytes(p.H);
  float s = 0.f;
  for (int b = lane; b < (int)mx_blocks(p.H); b += 64) {
    const u32x4 xc = *reinterpret_cast<const u32x4*>(a.x.codes + row * code_ld + 16l * b);
    const u32x4 wc = *reinterpret_cast<const u32x4*>(a.w.codes + t * code_ld + 16l * b);
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float xv[8], wv[8];
      mx_decode<kMxFp4>(u32x2_t{xc[i], 0u}, 127u, xv);
      mx_decode<kMxFp4>(u32x2_t{wc[i], 0u}, 127u, wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) d = fmaf(xv[j], wv[j], d);
    }
    const float sx = mx_scale(a.x.scales[row * scale_ld + b]);
    const float sw = mx_scale(a.w.scales[t * scale_ld + b]);
    s = fmaf(d * sx, sw, s);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
  if (lane == 0) p.zt[row] = s * p.scale;
}

template <class T>
void stream_logits(const MxLogitsArgs& a, hipStream_t s) {
  const int tb = a.M <= 32 ? 1 : a.M <= 64 ? 2 : 4;
  const unsigned g = (unsigned)(((int64_t)a.M + 32 * tb - 1) / (32 * tb) * a.n_vt);
  const int n = 64 * STREAM_WAVES;
  if (tb == 1) mx_stream_logits_kernel<T, 1><<<g, n, 0, s>>>(a);
  else if (tb == 2) mx_stream_logits_kernel<T, 2><<<g, n, 0, s>>>(a);
  else mx_stream_logits_kernel<T, 4><<<g, n, 0, s>>>(a);
}

template <bool ENT>
void stream_fwd(const MxFwdArgs& a, hipStream_t s) {
  const int tb = a.f.M <= 32 ? 1 : a.f.M <= 64 ? 2 : 4;
  const unsigned g = (unsigned)(((int64_t)a.f.M + 32 * tb - 1) / (32 * tb) * a.f.n_vt);
  const int n = 64 * STREAM_WAVES;
  if (tb == 1) mx_stream_fwd_kernel<1, ENT><<<g, n, 0, s>>>(a);
  else if (tb == 2) mx_stream_fwd_kernel<2, ENT><<<g, n, 0, s>>>(a);
  else mx_stream_fwd_kernel<4, ENT><<<g, n, 0, s>>>(a);
}

}  // namespace

hipError_t launch_mx_logits(const MxLogitsArgs& a, hipStream_t s) {
  if (a.out_dtype == kBf16) stream_logits<Bf16>(a, s);
  else stream_logits<F32>(a, s);
  return hipGetLastError();
}

hipError_t launch_mx_fwd_tile(const MxFwdArgs& a, bool entropy, hipStream_t s) {
  if (entropy) stream_fwd<true>(a, s);
  else stream_fwd<false>(a, s);
  return hipGetLastError();
}

hipError_t launch_mx_target_logit(const MxFwdArgs& a, hipStream_t s) {
  const unsigned g = (unsigned)(((long)a.f.M + TL_ROWS - 1) / TL_ROWS);
  mx_target_logit_kernel<<<g, 64 * TL_ROWS, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace flce
