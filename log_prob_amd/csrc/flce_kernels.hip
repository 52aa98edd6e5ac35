// HIP kernels of libflce for gfx950 (CDNA4): fused LM-head linear + cross-entropy.
//
// Forward (Liger-Kernel FSLCE commit, "Summary" and "Implementation / Forward";
// SkyRL PR 2141, "Overview"):
//   fwd_tile     one workgroup per (256-row M tile, 256-column V tile): bf16 MFMA
//                mainloop over H computing the tile transposed (vocabulary rows,
//                token columns), then an epilogue that reduces it to per-row partial
//                statistics (max m, sum of exp(z - m), and sum of exp(z - m) (z - m)
//                for entropy) down each lane's registers.
//   target_logit z[m, t[m]] as one dot product per row.
//   fwd_merge    combines the per-tile partials of each row (max first, then the
//                rescaled sums) into lse, logprob and entropy.
// Scalar reductions: nll_reduce (sum, count and mean of -logprob over valid rows) and
// nll_mean_grad (the mean NLL's gradient with respect to logprob); policy_loss_reduce
// and policy_loss_grad (a clipped policy-gradient loss on the log-probs, token-mean
// aggregated, and its gradient with respect to logprob).
// Backward (Liger-Kernel PR 1294, "Kernel design notes": recompute the logits
// tiles, emit d-logits in the input dtype into a reusable buffer, then two grad
// GEMMs; SkyRL PR 2141, "Overview": split backward over the vocabulary):
//   bwd_dlogits  the same mainloop on the same transposed tile, epilogue forms
//                scale * dz in bf16 for one vocabulary chunk, stored tile-blocked
//                (256 x 64 blocks).
//   gemm_dw      dW[chunk] = dz_chunk^T X          (K = tokens)
//   gemm_dx      dX (+)= dz_chunk W[chunk]          (K = chunk columns)
//
// Every kernel computes 256 x 256 output tiles with 4 waves of 128 x 128 and
// v_mfma_f32_32x32x16_bf16.  K is staged 64 at a time through double-buffered LDS
// (2 x 64 KiB) by direct-to-LDS buffer loads: no staging registers, and lanes whose
// 16 bytes lie outside the operand get an out-of-range offset, which the buffer
// unit turns into zeros.  An operand whose K dimension is contiguous in memory is
// kept in LDS as 128-byte K rows and read with ds_read_b128; an operand whose M/N
// dimension is contiguous is kept as 512-byte K rows and read with the gfx950
// transposing read ds_read_b64_tr_b16, which hands each lane 4 consecutive K values
// of one column.  Both layouts XOR-swizzle 16- or 32-byte blocks by row so the
// fragment reads are free of bank conflicts.  Kernels and the host code take a
// vocabulary offset, so the same kernels serve one shard of a split vocabulary.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>
#include <utility>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>
#include <utility>

#include "flce_internal.h"
#include "mainloop_device.h"
#include "tile_device.h"

namespace flce {

// The backward kernels run BigShape; their epilogues stage a 256 x 256 bf16 output
// tile (128 KiB) in the LDS the pipeline used.
constexpr int TILE = BigShape::TM;
constexpr int LDS_OUT = 2 * TILE * TILE;
constexpr int LDS_BIG = BigShape::PIPE_BYTES > LDS_OUT ? BigShape::PIPE_BYTES : LDS_OUT;
static_assert(BigShape::TN == TILE, "backward tile");

// ---------------------------------------------------------------------------
// bf16 output tiles of the backward kernels are staged in LDS before 16-byte
// coalesced stores.  Staging layout of a 256 x 256 tile: row r at byte 512 r, its
// 16-byte chunk c (columns 8 c .. 8 c + 7) at chunk position c ^ out_swz(r).  The
// swizzle sends the four rows one pair write touches (r0, r0 + 1, r0 + 4, r0 + 5,
// r0 even within its group of 8) to four different 64-byte bank groups.  Each wave
// stages its own 128 x 128 block and stores it 32 rows (one block row mb) at a time,
// right after staging them: no other wave touches those bytes, so no workgroup
// barrier, and the stores overlap the staging of the next block row.  The stores carry
// the non-temporal hint: no tile re-reads what it writes, and the lines would
// otherwise displace operand tiles in L2 (backward -0.7% at H = 2048, neutral at 8192).
__device__ __forceinline__ int out_swz(int r) { return ((r & 1) | ((r >> 1) & 2)) << 2; }

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Staging of values in the accumulator layout (element e of block (mb, nb) is row
// wr0 + 32 mb + acc_row(lane, e), column wc0 + 32 nb + lane % 32) as bf16 pairs.
// Lanes 2i and 2i + 1 hold adjacent columns of the same rows; a lane's rows r, r + 1
// (slots e = 4 q + jp, jp + 1 with jp in {0, 2}) are packed as one bf16x2 (row r
// low), exchanged with the partner lane by a DPP swap, and one byte permute keeps the
// even lane's row r (columns c, c + 1) and the odd lane's row r + 1 (c - 1, c); the
// conversion rounds to nearest even.  The rows a lane writes are r = wr0 + 32 mb +
// 8 q + 4 (lane / 32) + jp + (lane & 1), so out_swz(r) = 4 ((lane & 1) | 2 (lane /
// 32)) for all of them: one address per column block nb, and the row offsets
// 512 (32 mb + 8 q + jp) are immediates.
struct WaveStager {
  LDS_AS char* t3;
  uint32_t addr[4];
  uint32_t sel;  // v_perm_b32 byte selector: bytes 0-3 this lane's pair, 4-7 the partner's
  int wr0, wc0, lane;

  __device__ __forceinline__ void init(char* tile, int wr0_, int wc0_, int lane_) {
    wr0 = wr0_;
    wc0 = wc0_;
    lane = lane_;
    const int lc = lane & 31, hi = lane >> 5, odd = lane & 1;
    const int sw = odd | (hi << 1);
    t3 = (LDS_AS char*)tile;
    const uint32_t base =
        (uint32_t)((wr0 + 4 * hi + odd) * 512 + (wc0 >> 3) * 16 + (lc & 6) * 2);
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) addr[nb] = base + (uint32_t)((((nb ^ sw) << 2) + (lc >> 3)) << 4);
    sel = odd ? 0x03020706u : 0x05040100u;
  }

  // v0, v1: this lane's values in slots e = 4 q + jp and 4 q + jp + 1 of block (mb, nb)
  __device__ __forceinline__ void put(int mb, int q, int jp, int nb, float v0, float v1) const {
    const f32x2 pr = {v0, v1};
    const uint32_t own = __builtin_bit_cast(uint32_t, __builtin_convertvector(pr, bf16x2));
    const uint32_t partner = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)own, 0xB1, 0xf, 0xf, true);
    *(LDS_AS uint32_t*)(t3 + addr[nb] + (32 * mb + 8 * q + jp) * 512) =
        __builtin_amdgcn_perm(partner, own, sel);
  }

  // The 16 bytes of tile row r, chunk c (columns 8 c .. 8 c + 7).
  __device__ __forceinline__ u32x4 get(int r, int c) const {
    return *(LDS_AS const u32x4*)(t3 + r * 512 + ((c ^ out_swz(r)) << 4));
  }

  // Wait until this wave's staging writes are in LDS (its own reads follow).
  __device__ __forceinline__ void fence() const { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

  // Store the wave's staged rows of block row mb to rows [0, nrows) and columns
  // [0, ncols) of a row-major matrix (dst = the tile's element (0, 0), leading
  // dimension ld; ncols a multiple of 8): 4 rows of 256 bytes per instruction.
  __device__ __forceinline__ void store_rows(int mb, uint16_t* dst, long ld, int nrows,
                                             int ncols) const {
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      const int r = wr0 + 32 * mb + 4 * it + (lane >> 4), c = (wc0 >> 3) + (lane & 15);
      const u32x4 v = get(r, c);
      if (r < nrows && 8 * c < ncols)
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(dst + (long)r * ld + 8 * c));
    }
  }
};

// A wave's 128 x 128 accumulator block rounded to bf16 and stored to rows [0, nrows)
// and columns [0, ncols) of a row-major matrix (dst = the tile's element (0, 0)).
__device__ __forceinline__ void store_acc_bf16(char* tile, const f32x16 (&acc)[4][4], int wr0,
                                               int wc0, int lane, uint16_t* dst, long ld,
                                               int nrows, int ncols) {
  WaveStager st;
  st.init(tile, wr0, wc0, lane);
#pragma unroll
  for (int mb = 0; mb < 4; ++mb) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int jp = 0; jp < 4; jp += 2)
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
          st.put(mb, q, jp, nb, acc_read(acc[mb][nb][4 * q + jp]),
                 acc_read(acc[mb][nb][4 * q + jp + 1]));
    st.fence();
    st.store_rows(mb, dst, ld, nrows, ncols);
  }
}

// ---------------------------------------------------------------------------
// Forward tile kernel.

// One workgroup per tile of TN tokens x TM vocabulary entries of the logits, computed
// transposed (z^T = W X^T) and reduced to the tokens' partials by fwd_epilogue.
template <class S, bool ENT>
__global__ __launch_bounds__(S::NTHREADS, S::WAVES_PER_EU) void fwd_tile_kernel(FwdTileArgs p) {
  constexpr int TV = S::TM, TT = S::TN;
  __shared__ __attribute__((aligned(1024))) char smem[S::PIPE_BYTES];
  int mt, vt;
  {
    const int L = tile_claim(p.n_mt * p.n_vt, p.tq);
    if (L < 0) return;
    group_coords(L, p.n_mt, p.n_vt, FWD_GROUP_M, mt, vt);
  }
  const int row0 = mt * TT, col0 = vt * TV;  // first token, first vocabulary entry

  f32x16 acc[S::MB][S::NB];
  const TileSrc A{p.W + (long)col0 * p.H, p.H, p.V - col0, p.H, 0};
  const TileSrc B{p.X + (long)row0 * p.H, p.H, p.M - row0, p.H, 0};
  mainloop<S, true, true, true>(acc, smem, A, B, p.H);  // X (L2-resident) loads first
  // (the mainloop ends with a barrier: the LDS is free)
  fwd_epilogue<S, ENT>(acc, smem, p, mt, vt);
}

// Target logit of every row whose target W holds: z[m, t[m]] = scale * X[m] . W[t[m] -
// v_off], bf16 products accumulated in fp32 in a fixed order (each lane over a strided
// set of 8-element groups, then a fixed butterfly over the wave).  A separate pass
// rather than a pick in the tile epilogue: the pick would have to run in every wave
// of every tile (a tile that picks only where a target lies costs more than the others
// and breaks the lockstep of an XCD's tiles), which took a quarter of the epilogue.
// One wave per row.
constexpr int TL_ROWS = 4;
__global__ __launch_bounds__(64 * TL_ROWS) void target_logit_kernel(FwdTileArgs p) {
  // zero the tile kernel's queue counters: that kernel is launched after this one
  if (blockIdx.x == 0 && threadIdx.x < 8 && p.tq.ctr)
    __hip_atomic_store(&p.tq.ctr[threadIdx.x], 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const int lane = threadIdx.x & 63;
  const long row = (long)blockIdx.x * TL_ROWS + (threadIdx.x >> 6);
  if (row >= p.M) return;
  const int64_t t = p.targets[row];
  const int64_t tw = t - p.v_off;
  if (t == p.ignore_index || tw < 0 || tw >= p.V) return;
  const uint16_t* x = p.X + row * p.H;
  const uint16_t* w = p.W + tw * p.H;
  float s = 0.f;
#pragma unroll 4
  for (int k = 8 * lane; k < p.H; k += 8 * 64) {
    const u32x4 xv = *reinterpret_cast<const u32x4*>(x + k);
    const u32x4 wv = *reinterpret_cast<const u32x4*>(w + k);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s = fmaf(__uint_as_float(xv[i] << 16), __uint_as_float(wv[i] << 16), s);
      s = fmaf(__uint_as_float(xv[i] & 0xffff0000u), __uint_as_float(wv[i] & 0xffff0000u), s);
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
  if (lane == 0) p.zt[row] = s * p.scale;
}

// Merge of the per-tile partials of each row: m* = max m_j, S = sum s_j e^(m_j - m*),
// U = sum e^(m_j - m*) (u_j + (m_j - m*) s_j); lse = m* + log S,
// logprob = min(z_t - lse, 0), entropy = max(log S - U / S, 0).
// The tiles j run over every shard of the table in order (one shard when the
// vocabulary is not split); the target logit comes from the shard that owns the target.
// A workgroup takes MERGE_ROWS rows; its MERGE_SLICES slices split each row's tiles
// (32 lanes read consecutive rows of one tile, so every load is a 128-byte line) and
// combine their maxima, then their sums, through LDS.  32 rows x 16 slices measured
// faster than 64 x 8 (fewer tiles per thread, twice the workgroups: 35 -> 22 us at
// M = H = 8192, V = 131072) and than 16 x 32 (64-byte pieces).
constexpr int MERGE_ROWS = 32, MERGE_SLICES = 16;
template <bool ENT>
__global__ __launch_bounds__(MERGE_ROWS * MERGE_SLICES) void fwd_merge_kernel(FwdMergeArgs p) {
  __shared__ float sm[3][MERGE_SLICES][MERGE_ROWS];
  const int lr = threadIdx.x % MERGE_ROWS, sl = threadIdx.x / MERGE_ROWS;
  const int row = blockIdx.x * MERGE_ROWS + lr;
  const bool live = row < p.M;
  float m = -INFINITY;
  if (live)
    for (int r = 0; r < p.sh.n; ++r) {
      const float* pm = p.base + p.sh.part_m[r] + row;
      for (int j = sl; j < p.sh.n_vt[r]; j += MERGE_SLICES) m = fmaxf(m, pm[(long)j * p.Mpad]);
    }
  sm[0][sl][lr] = m;
  __syncthreads();
  float ms = -INFINITY;
#pragma unroll
  for (int k = 0; k < MERGE_SLICES; ++k) ms = fmaxf(ms, sm[0][k][lr]);
  float S = 0.f, U = 0.f;
  if (live)
    for (int r = 0; r < p.sh.n; ++r) {
      const float* pm = p.base + p.sh.part_m[r] + row;
      const float* ps = p.base + p.sh.part_s[r] + row;
      const float* pu = p.base + p.sh.part_u[r] + row;
      for (int j = sl; j < p.sh.n_vt[r]; j += MERGE_SLICES) {
        const long off = (long)j * p.Mpad;
        const float dm = pm[off] - ms;
        const float a = __expf(dm);
        const float s = ps[off];
        S += s * a;
        if constexpr (ENT) U += a * (pu[off] + dm * s);
      }
    }
  sm[1][sl][lr] = S;
  sm[2][sl][lr] = U;
  __syncthreads();
  if (sl != 0 || !live) return;
  S = 0.f;
  U = 0.f;
#pragma unroll
  for (int k = 0; k < MERGE_SLICES; ++k) {
    S += sm[1][k][lr];
    if constexpr (ENT) U += sm[2][k][lr];
  }
  const float logS = log_sum(S);
  const int64_t t = p.targets[row];
  const bool valid = t != p.ignore_index && t >= 0 && t < p.sh.v_lo[p.sh.n];
  float zt = 0.f;
  if (valid) {
    int r = 0;
    while (r + 1 < p.sh.n && t >= p.sh.v_lo[r + 1]) ++r;
    zt = p.base[p.sh.zt[r] + row];
  }
  p.lse[row] = ms + logS;
  // A log-probability is at most 0 and an entropy at least 0.  When one logit holds
  // nearly all of a row's probability both values sit next to that bound, and fp32
  // rounding can put them a few ulps past it: the target logit (its own dot product)
  // and lse (from the MFMA accumulators) round differently, and the shifted sum of the
  // row's maximum element can come out a hair above 0.  The bounds are applied
  // exactly, which only moves a value towards the true one; a NaN passes them.
  p.logprob[row] = valid ? at_most_zero(zt - (ms + logS)) : 0.f;
  if constexpr (ENT) p.entropy[row] = valid ? at_least_zero(logS - U / S) : 0.f;
}

// ---------------------------------------------------------------------------
// Staging of a d-logit tile computed transposed (vocabulary rows, token columns in the
// accumulators) for the tile-blocked buffer: token row r of the 256 x 256 bf16 tile at
// byte 512 r, its 16-byte chunk c (vocabulary columns 8 c .. 8 c + 7) at chunk
// position c ^ tswz(r).  A staging write puts 4 consecutive vocabulary entries of 32
// consecutive token rows, all in one chunk, and tswz is a bijection of r % 32, so the
// 64 lanes' 8-byte pieces fill 32 distinct chunk positions; a store read takes 8
// consecutive chunks of 4 consecutive rows per 32 lanes, which tswz (r % 4 in its top
// bits) sends to 4 distinct groups of 8 positions.  Both are free of bank conflicts
// (128 banks), and each wave's bytes are its own.
__device__ __forceinline__ int tswz(int r) { return ((r & 3) << 3) | ((r >> 2) & 7); }

struct DzStager {
  LDS_AS char* t3;
  uint32_t row[4];  // byte offset of token row wt0 + 32 nb + lane % 32
  int sw[4];
  int wt0, wv0, lane;

  __device__ __forceinline__ void init(char* tile, int wt0_, int wv0_, int lane_) {
    wt0 = wt0_;
    wv0 = wv0_;
    lane = lane_;
    t3 = (LDS_AS char*)tile;
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      const int r = wt0 + 32 * nb + (lane & 31);
      row[nb] = (uint32_t)r * 512u + (uint32_t)(lane >> 5) * 8u;
      sw[nb] = tswz(r);
    }
  }

  // vocabulary rows wv0 + 32 mb + 8 q + 4 (lane / 32) + 0..3 of token column nb
  __device__ __forceinline__ void put(int nb, int mb, int q, const float (&d)[4]) const {
    const int c = (wv0 >> 3) + 4 * mb + q;
    const f32x2 p0 = {d[0], d[1]}, p1 = {d[2], d[3]};
    const u32x2 v = {__builtin_bit_cast(uint32_t, __builtin_convertvector(p0, bf16x2)),
                     __builtin_bit_cast(uint32_t, __builtin_convertvector(p1, bf16x2))};
    *(LDS_AS u32x2*)(t3 + row[nb] + ((c ^ sw[nb]) << 4)) = v;
  }

  // Wait until this wave's staging writes are in LDS (its own reads follow).
  __device__ __forceinline__ void fence() const { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

  // Store the wave's staged token rows of block nb (32 rows, its 128 vocabulary
  // columns) to the tile-blocked buffer (dst = the tile's 256 x 64 block 0, block q at
  // dst + q BLK_ELEMS, row r at 64 r): two pieces of 32 consecutive rows, 1 KiB per
  // instruction.
  __device__ __forceinline__ void store_blocked(int nb, uint16_t* dst) const {
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      const int qb = it >> 2, r = wt0 + 32 * nb + 8 * (it & 3) + (lane >> 3), c8 = lane & 7;
      const int c = (wv0 >> 3) + 8 * qb + c8;
      const u32x4 v = *(LDS_AS const u32x4*)(t3 + r * 512 + ((c ^ tswz(r)) << 4));
      __builtin_nontemporal_store(
          v, reinterpret_cast<u32x4*>(dst + (long)((wv0 >> 6) + qb) * BLK_ELEMS + r * BLK_COLS + 8 * c8));
    }
  }
};

// A wave's d-logits, d = 2^(c1 acc - lse2) (c0 + cb acc) + [row = target] sa with the
// per-token parameters of its 4 token columns (from LDS, see bwd_dlogits_kernel),
// rounded to bf16, staged in the wave's own part of the LDS tile and stored to the
// tile-blocked buffer at dst (the tile's 256 x 64 block 0) 32 token rows at a time.
// RAGGED: vocabulary rows at or past `vrows` of the wave tile become 0.  Every wave
// runs the same instruction stream whether or not it holds a target (the correction is
// a branch per four vocabulary rows that almost never has active lanes), which keeps
// the tiles of an XCD in step.
template <bool ENTGRAD, bool RAGGED>
__device__ __forceinline__ void stage_dlogits(char* tile, const f32x16 (&acc)[4][4],
                                              const float* r_lse2, const float* r_c0,
                                              const float* r_cb, const float* r_sa,
                                              const int* t_local, int wv0, int wt0, int lane,
                                              float c1, int vrows, uint16_t* dst) {
  const int lc = lane & 31, hi = lane >> 5;
  float L[4], C0[4], CB[4], SA[4];
  int T[4];
#pragma unroll
  for (int nb = 0; nb < 4; ++nb) {
    const int t = wt0 + 32 * nb + lc;
    L[nb] = r_lse2[t];
    C0[nb] = r_c0[t];
    CB[nb] = ENTGRAD ? r_cb[t] : 0.f;
    SA[nb] = r_sa[t];
    T[nb] = t_local[t] - wv0 - 4 * hi;  // the target's row among the lane's, if any
  }
  DzStager st;
  st.init(tile, wt0, wv0, lane);
#pragma unroll
  for (int nb = 0; nb < 4; ++nb) {
#pragma unroll
    for (int mb = 0; mb < 4; ++mb)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float d[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float av = acc_read(acc[mb][nb][4 * q + j]);
          const float pr = __builtin_amdgcn_exp2f(fmaf(av, c1, -L[nb]));
          float v = pr * (ENTGRAD ? fmaf(CB[nb], av, C0[nb]) : C0[nb]);
          if constexpr (RAGGED) v = 32 * mb + 8 * q + 4 * hi + j < vrows ? v : 0.f;
          d[j] = v;
        }
        const int dd = T[nb] - 32 * mb - 8 * q;
        if ((unsigned)dd < 4u) {
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] += dd == j ? SA[nb] : 0.f;
        }
        st.put(nb, mb, q, d);
      }
    st.fence();
    st.store_blocked(nb, dst);
  }
}

// Backward d-logits for one vocabulary chunk: dzs = scale * dz in bf16, written to
// an Mpad x ldz tile-blocked buffer (chunk column j = vocabulary column vbase + j;
// 256-row bands of 256 x 64 blocks, so that the GEMMs that read it take contiguous
// 32 KiB blocks instead of 128-byte pieces of 256 KiB-apart rows).  Columns past
// V and rows past M are written as zero.  With p = 2^(c1 acc - lse2) (c1 = scale log2 e)
// and per-row a = grad_logprob, b = grad_entropy, E = lse - entropy (all 0 on ignored
// rows):  scale dz = scale (a ([v = t] - p) + b p (E - scale acc))
//                  = p (c0 + cb acc) + [v = t] sa,
// c0 = scale (b E - a), cb = -scale^2 b, sa = scale a.
// LDS of the d-logit tile: the pipeline, then the bf16 output tile and the per-row arrays
constexpr int LDS_DLOGITS = BigShape::PIPE_BYTES > LDS_OUT + 5 * TILE * 4
                                ? BigShape::PIPE_BYTES
                                : LDS_OUT + 5 * TILE * 4;

template <bool ENTGRAD>
__device__ __forceinline__ void dlogits_tile(const DlogitsArgs& p, int mt, int vt, char* smem) {
  const int row0 = mt * TILE, ccol0 = vt * TILE, col0 = p.vbase + ccol0;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // wave-uniform
  // row tid's parameters, kept in registers over the mainloop (which may need all of
  // the LDS) and published through LDS after it
  float lse2 = 0.f, c0 = 0.f, cb = 0.f, sa = 0.f;
  int tl = -1;
  {
    const int r = row0 + tid;
    if (r < p.M) {
      // all of the row's loads go out together (validity selects afterwards, so no
      // load waits for the target's): one round trip, under the mainloop's first loads
      const int64_t t = p.targets[r];
      const float lse = p.lse[r];
      const float a = p.grad_logprob ? p.grad_logprob[r] : 0.f;
      float b = 0.f, ent = 0.f;
      if constexpr (ENTGRAD) {
        b = p.grad_entropy[r];
        ent = p.entropy[r];
      }
      const bool valid = t != p.ignore_index && t >= 0 && t < p.V_total;
      const int64_t tw = t - p.v_off;  // target as a row of W (owned iff 0 <= tw < V)
      lse2 = lse * LOG2E;
      const float sa_r = p.scale * a;
      const float c0_r = ENTGRAD ? p.scale * (b * (lse - ent) - a) : -sa_r;
      const float cb_r = ENTGRAD ? -p.scale * p.scale * b : 0.f;
      sa = valid ? sa_r : 0.f;
      c0 = valid ? c0_r : 0.f;
      cb = valid ? cb_r : 0.f;
      tl = (valid && tw >= col0 && tw < col0 + TILE && tw < p.V) ? (int)(tw - col0) : -1;
    }
  }

  // the tile computed transposed: vocabulary rows (A = W), token columns (B = X, whose
  // loads go first in each stage)
  f32x16 acc[4][4];
  const TileSrc A{p.W + (long)col0 * p.H, p.H, p.V - col0, p.H, 0};
  const TileSrc B{p.X + (long)row0 * p.H, p.H, p.M - row0, p.H, 0};
  mainloop<BigShape, true, true, true>(acc, smem, A, B, p.H);

  float* r_lse2 = reinterpret_cast<float*>(smem + LDS_OUT);
  float* r_c0 = r_lse2 + TILE;
  float* r_cb = r_c0 + TILE;
  float* r_sa = r_cb + TILE;
  int* t_local = reinterpret_cast<int*>(r_sa + TILE);
  r_lse2[tid] = lse2;
  r_c0[tid] = c0;
  if constexpr (ENTGRAD) r_cb[tid] = cb;
  r_sa[tid] = sa;
  t_local[tid] = tl;
  __syncthreads();

  const int wv0 = (wave >> 1) * 128, wt0 = (wave & 1) * 128;
  const float c1 = p.scale * LOG2E;
  const bool ragged = col0 + TILE > p.V;
  const int vrows = p.V - col0 - wv0;  // vocabulary rows of the wave tile that exist
  uint16_t* const dst = p.dz + (long)mt * BLK_ROWS * p.ldz + (long)(ccol0 / BLK_COLS) * BLK_ELEMS;
  if (!ragged)
    stage_dlogits<ENTGRAD, false>(smem, acc, r_lse2, r_c0, r_cb, r_sa, t_local, wv0, wt0, lane, c1,
                                  vrows, dst);
  else
    stage_dlogits<ENTGRAD, true>(smem, acc, r_lse2, r_c0, r_cb, r_sa, t_local, wv0, wt0, lane, c1,
                                 vrows, dst);
}

template <bool ENTGRAD>
__global__ __launch_bounds__(NTHREADS) void bwd_dlogits_kernel(DlogitsArgs p) {
  __shared__ __attribute__((aligned(1024))) char smem[LDS_DLOGITS];
  const int L = tile_claim(p.n_mt * p.n_vt, p.tq);
  if (L < 0) return;
  int mt, vt;
  group_coords(L, p.n_mt, p.n_vt, 8, mt, vt);
  dlogits_tile<ENTGRAD>(p, mt, vt, smem);
}

// ---------------------------------------------------------------------------
// The fp32 side of an output tile (modes 1-3), for dX across vocabulary chunks and dW
// across token waves.  t.acc and t.out point at the tile's element (0, 0) of an fp32
// accumulator and of the bf16 result, both with leading dimension t.ld; rows
// [0, t.nrows) and columns [0, t.ncols) of the tile exist.  Each wave moves its
// 128 x 128 block through a private 32 KiB LDS slice, 64 rows at a time, so the fp32
// accumulator is read and written in 16-byte pieces (a half-wave covers 512 contiguous
// bytes of a row) and all of a lane's loads of a slice are in flight together;
// per-element accesses in the accumulator layout would wait on one read-modify-write
// after another.  Slice layout: row r (0..63) at 512 r bytes, column c at float
// (c ^ 32 ((r >> 2) & 1)), so the two half-waves of a staging write (rows r and r + 4)
// fall on different banks.
// mode 1: acc = v; mode 2: acc += v; mode 3: out = bf16(acc + v).
struct F32Tile {
  float* acc;
  uint16_t* out;
  long ld;
  int nrows, ncols;
  int mode;
};

__device__ __forceinline__ void tile_f32(const f32x16 (&acc)[4][4], char* smem, const F32Tile& t,
                                         int wave, int lane) {
  const int wr0 = (wave >> 1) * 128, wc0 = (wave & 1) * 128;
  float* sl = reinterpret_cast<float*>(smem + wave * 32768);
  const int lc = lane & 31, hi = lane >> 5;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int mi = 0; mi < 2; ++mi)
#pragma unroll
      for (int nb = 0; nb < 4; ++nb)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int r = 32 * mi + acc_row(lane, e);  // (r >> 2) & 1 == hi
          sl[r * 128 + ((32 * nb + lc) ^ (hi << 5))] = acc_read(acc[2 * s + mi][nb][e]);
        }
    __syncthreads();
    const int rb = wr0 + 64 * s, cb = wc0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      // granule g = 64 it + lane: row g / 32, columns 4 (g % 32) .. + 3
      float4 old[16];
#pragma unroll
      for (int it = 0; it < 16; ++it) {
        const int g = 64 * (16 * half + it) + lane, r = g >> 5, c = 4 * (g & 31);
        const int m = rb + r, h = cb + c;
        old[it] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t.mode != 1 && m < t.nrows && h < t.ncols)
          old[it] = *reinterpret_cast<const float4*>(t.acc + (long)m * t.ld + h);
      }
#pragma unroll
      for (int it = 0; it < 16; ++it) {
        const int g = 64 * (16 * half + it) + lane, r = g >> 5, c = 4 * (g & 31);
        const int m = rb + r, h = cb + c;
        const float4 v = *reinterpret_cast<const float4*>(sl + r * 128 + (c ^ (((r >> 2) & 1) << 5)));
        const float4 u = t.mode == 1 ? v
                                     : make_float4(old[it].x + v.x, old[it].y + v.y,
                                                   old[it].z + v.z, old[it].w + v.w);
        if (m < t.nrows && h < t.ncols) {
          if (t.mode == 3) {
            const f32x2 lo = {u.x, u.y}, hi2 = {u.z, u.w};
            const uint32_t a = __builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2));
            const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_convertvector(hi2, bf16x2));
            *reinterpret_cast<uint2*>(t.out + (long)m * t.ld + h) = make_uint2(a, b);
          } else {
            __builtin_nontemporal_store(__builtin_bit_cast(u32x4, u),
                                        reinterpret_cast<u32x4*>(t.acc + (long)m * t.ld + h));
          }
        }
      }
    }
    __syncthreads();
  }
}

// dW[vbase + i, h] = sum_m dzs[m, i] X[m, h]: A = dzs^T (MN), B = X^T (MN), K = Mpad.
// mode 0: write bf16; 1-3: the fp32 accumulator across token waves (see tile_f32).
__device__ __forceinline__ void dw_tile(const GemmDwArgs& p, int ti, int th, char* smem) {
  const int i0 = ti * TILE, h0 = th * TILE;
  f32x16 acc[4][4];
  // dzs has Mpad rows (rows past M hold zeros); X has only M rows.
  const TileSrc A{p.dz + (long)(i0 / BLK_COLS) * BLK_ELEMS, BLK_COLS, p.chunk_cols - i0, p.Mpad,
                  (long)BLK_ROWS * p.ldz};
  const TileSrc B{p.X + h0, p.H, p.H - h0, p.M, 0};
  // the X^T loads (L2-resident) go out before the streamed d-logit loads of each step
  mainloop<BigShape, false, false, true>(acc, smem, A, B, p.Mpad);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wr0 = (wave >> 1) * 128, wc0 = (wave & 1) * 128;
  const int rows = min(min(TILE, p.chunk_cols - i0), p.V - (p.vbase + i0));
  const long o = (long)(p.vbase + i0) * p.H + h0;
  if (p.mode == 0)
    store_acc_bf16(smem, acc, wr0, wc0, lane, p.dW + o, p.H, rows, p.H - h0);
  else
    tile_f32(acc, smem, F32Tile{p.acc + o, p.dW + o, p.H, rows, p.H - h0, p.mode}, wave, lane);
}

__global__ __launch_bounds__(NTHREADS) void gemm_dw_kernel(GemmDwArgs p) {
  __shared__ __attribute__((aligned(1024))) char smem[LDS_BIG];
  const int L = tile_claim(p.n_h * p.n_i, p.tq);
  if (L < 0) return;
  int ti, th;
  // groups run along H: the few X^T tiles stay in L2 while each dzs tile is read by
  // one group of an XCD at a time, so dzs streams from HBM about once per H group
  group_coords(L, p.n_h, p.n_i, 8, th, ti);
  dw_tile(p, ti, th, smem);
}

// dX[m, h] (+)= sum_i dzs[m, i] W[vbase + i, h]: A = dzs (KC), B = W^T (MN), K = kcols.
// mode 0: write bf16; 1: write fp32 accumulator; 2: accumulate fp32; 3: accumulate and write bf16.
__device__ __forceinline__ void dx_tile(const GemmDxArgs& p, int tm, int th, char* smem) {
  const int m0 = tm * TILE, h0 = th * TILE;
  f32x16 acc[4][4];
  // the chunk's kcols (padded) columns of dzs (band tm of the blocked buffer); W has
  // V - vbase rows left
  const long band = (long)BLK_ROWS * p.ldz;
  const TileSrc A{p.dz + (long)tm * band, BLK_COLS, p.M - m0, p.kcols, band};
  const TileSrc B{p.W + (long)p.vbase * p.H + h0, p.H, p.H - h0, p.V - p.vbase, 0};
  mainloop<BigShape, true, false>(acc, smem, A, B, p.kcols);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wr0 = (wave >> 1) * 128, wc0 = (wave & 1) * 128;
  if (p.mode == 0) {
    store_acc_bf16(smem, acc, wr0, wc0, lane, p.dX + (long)m0 * p.H + h0, p.H, p.M - m0,
                   p.H - h0);
  } else {
    const long o = (long)m0 * p.H + h0;
    tile_f32(acc, smem, F32Tile{p.acc + o, p.dX + o, p.H, p.M - m0, p.H - h0, p.mode}, wave,
             lane);
  }
}

__global__ __launch_bounds__(NTHREADS) void gemm_dx_kernel(GemmDxArgs p) {
  __shared__ __attribute__((aligned(1024))) char smem[LDS_BIG];
  int tm, th;
  // groups run along H: in step, the XCDs read the same W columns (shared through the
  // memory-side cache) while each streams d-logit bands of its own
  tile_coords(blockIdx.x, gridDim.x, p.n_h, p.n_m, 8, th, tm);
  dx_tile(p, tm, th, smem);
}

// ---------------------------------------------------------------------------
// Pipelined backward: one launch runs the dW and dX tiles of one step (a token wave x
// vocabulary chunk, reading that step's d-logit buffer) together with the d-logit
// tiles of the next step (writing the other buffer), so no tile of a launch depends on
// another one, and the backward takes n + 1 launches for n steps instead of 3 n.  Each
// XCD (workgroup id modulo 8) takes an eighth of each kind of tile, contiguous in that
// kind's L2-grouped order, and works through its dW tiles first, then its dX tiles,
// then its d-logit tiles; ids past an XCD's share exit at once.
static_assert(LDS_DLOGITS >= LDS_BIG, "one LDS size serves every tile kind");

__device__ __forceinline__ void xcd_share(int n, int x, int& lo, int& cnt) {
  lo = (int)((long)n * x / 8);
  cnt = (int)((long)n * (x + 1) / 8) - lo;
}

template <bool ENTGRAD>
__global__ __launch_bounds__(NTHREADS) void bwd_pipe_kernel(PipeArgs p) {
  __shared__ __attribute__((aligned(1024))) char smem[LDS_DLOGITS];
  const int x = blockIdx.x & 7;
  int pos = blockIdx.x >> 3, lo, cnt;
  xcd_share(p.n_dw, x, lo, cnt);
  if (pos < cnt) {
    int ti, th;
    group_coords(lo + pos, p.dw.n_h, p.dw.n_i, 8, th, ti);
    dw_tile(p.dw, ti, th, smem);
    return;
  }
  pos -= cnt;
  xcd_share(p.n_dx, x, lo, cnt);
  if (pos < cnt) {
    int tm, th;
    group_coords(lo + pos, p.dx.n_h, p.dx.n_m, 8, th, tm);
    dx_tile(p.dx, tm, th, smem);
    return;
  }
  pos -= cnt;
  xcd_share(p.n_dl, x, lo, cnt);
  if (pos < cnt) {
    int mt, vt;
    group_coords(lo + pos, p.dl.n_mt, p.dl.n_vt, 8, mt, vt);
    dlogits_tile<ENTGRAD>(p.dl, mt, vt, smem);
  }
}

// Scalar cross-entropy reductions over the valid rows, in one workgroup so the order
// of every addition is fixed (bitwise repeatable): thread t takes rows t, t + 1024, ...
// in fp64, then a fixed tree over the threads.  out = {sum of -logprob, valid rows,
// mean (NaN without a valid row)}.
constexpr int NLL_THREADS = 1024;
__global__ __launch_bounds__(NLL_THREADS) void nll_reduce_kernel(const float* __restrict__ logprob,
                                                                 const int64_t* __restrict__ targets,
                                                                 long M, int64_t V,
                                                                 int64_t ignore_index,
                                                                 double* __restrict__ out) {
  __shared__ double ss[NLL_THREADS];
  __shared__ long sc[NLL_THREADS];
  const int t = threadIdx.x;
  double s = 0.0;
  long c = 0;
  for (long i = t; i < M; i += NLL_THREADS) {
    const int64_t tg = targets[i];
    if (tg != ignore_index && tg >= 0 && tg < V) {
      s -= (double)logprob[i];
      ++c;
    }
  }
  ss[t] = s;
  sc[t] = c;
  __syncthreads();
  for (int w = NLL_THREADS / 2; w > 0; w >>= 1) {
    if (t < w) {
      ss[t] += ss[t + w];
      sc[t] += sc[t + w];
    }
    __syncthreads();
  }
  if (t == 0) {
    out[0] = ss[0];
    out[1] = (double)sc[0];
    out[2] = sc[0] > 0 ? ss[0] / (double)sc[0] : __builtin_nan("");
  }
}

// grad[i] = -1 / n on valid rows (n = the valid-row count in reduced[1]), else 0.
__global__ void nll_mean_grad_kernel(const int64_t* __restrict__ targets, long M, int64_t V,
                                     int64_t ignore_index, const double* __restrict__ reduced,
                                     float* __restrict__ grad) {
  const double n = reduced[1];
  const float g = n > 0.0 ? (float)(-1.0 / n) : 0.f;
  const long stride = (long)gridDim.x * blockDim.x;
  for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < M; i += stride) {
    const int64_t tg = targets[i];
    grad[i] = (tg != ignore_index && tg >= 0 && tg < V) ? g : 0.f;
  }
}

// Clipped policy loss on the per-token log-probs (Liger-Kernel PR 1294, "Chunked Triton
// GRPO loss": the loss on top of the fused linear log-probs, with clip range and
// token-level normalisation; the page gives no formulas, the plain reading is the
// clipped surrogate).  Per valid token, in fp64: r = exp(logprob - old_logprob),
// c = min(max(r, 1 - eps_low), 1 + eps_high), loss = -min(r A, c A), clipped iff
// c A < r A.  Both kernels evaluate the same expression, so the gradient kernel takes
// the same clip decision as the reduction.
struct PolicyTerm {
  double u, cl;  // r A and c A
  bool valid;
};
__device__ __forceinline__ PolicyTerm policy_term(const PolicyLossArgs& p, long i) {
  PolicyTerm o;
  const int64_t tg = p.targets[i];
  o.valid = tg != p.ignore_index && tg >= 0 && tg < p.V;
  const double lp = (double)p.logprob[i];
  const double old = p.old_logprob ? (double)p.old_logprob[i] : lp;
  const double a = (double)p.advantages[i];
  const double r = exp(lp - old);
  // by comparisons, here and for the minimum: fmin and fmax would drop a NaN
  const double lo = 1.0 - p.eps_low, hi = 1.0 + p.eps_high;
  const double c = r < lo ? lo : r > hi ? hi : r;
  o.u = r * a;
  o.cl = c * a;
  return o;
}

// One workgroup, fixed summation order (bitwise repeatable): thread t takes tokens
// t, t + 1024, ..., then a fixed tree.  Writes the per-token loss (0 on invalid rows)
// and clip flags, and out = {sum of the loss, valid rows, clipped rows, sum / N} with
// N = denominator if > 0, else the valid rows (NaN when N is 0).
constexpr int PL_THREADS = 1024;
__global__ __launch_bounds__(PL_THREADS) void policy_loss_reduce_kernel(
    PolicyLossArgs p, float* __restrict__ per_token_loss, uint8_t* __restrict__ is_clipped,
    double* __restrict__ out) {
  __shared__ double ss[PL_THREADS];
  __shared__ long sn[PL_THREADS], sk[PL_THREADS];
  const int t = threadIdx.x;
  double s = 0.0;
  long n = 0, k = 0;
  for (long i = t; i < p.M; i += PL_THREADS) {
    const PolicyTerm o = policy_term(p, i);
    const bool clipped = o.valid && o.cl < o.u;
    const double loss = o.valid ? -(o.cl < o.u ? o.cl : o.u) : 0.0;
    per_token_loss[i] = (float)loss;
    if (is_clipped) is_clipped[i] = clipped ? 1 : 0;
    s += loss;
    n += o.valid ? 1 : 0;
    k += clipped ? 1 : 0;
  }
  ss[t] = s;
  sn[t] = n;
  sk[t] = k;
  __syncthreads();
  for (int w = PL_THREADS / 2; w > 0; w >>= 1) {
    if (t < w) {
      ss[t] += ss[t + w];
      sn[t] += sn[t + w];
      sk[t] += sk[t + w];
    }
    __syncthreads();
  }
  if (t == 0) {
    const double N = p.denominator > 0.0 ? p.denominator : (double)sn[0];
    out[0] = ss[0];
    out[1] = (double)sn[0];
    out[2] = (double)sk[0];
    out[3] = N > 0.0 ? ss[0] / N : __builtin_nan("");
  }
}

// grad[i] = -r A / N on valid tokens whose minimum takes the unclipped term, else 0;
// N as in the reduction (the valid-row count read from reduced[1] when the
// denominator is not positive).
__global__ void policy_loss_grad_kernel(PolicyLossArgs p, const double* __restrict__ reduced,
                                        float* __restrict__ grad) {
  const double N = p.denominator > 0.0 ? p.denominator : reduced[1];
  const long stride = (long)gridDim.x * blockDim.x;
  for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < p.M; i += stride) {
    const PolicyTerm o = policy_term(p, i);
    grad[i] = (o.valid && !(o.cl < o.u) && N > 0.0) ? (float)(-o.u / N) : 0.f;
  }
}

__global__ void fill_u16_kernel(uint16_t* __restrict__ p, long n) {
  const long i = (long)blockIdx.x * blockDim.x + threadIdx.x;
  const long stride = (long)gridDim.x * blockDim.x;
  for (long j = i; j < n; j += stride) p[j] = 0;
}

// ---------------------------------------------------------------------------
// Scratch of the allocation-free forward: the partials of its token waves.  A
// __device__ array is module memory: each GPU the library runs on holds its own copy,
// at its own address, from the module's load until the process ends.  In host code
// `scratch` names a host-side stand-in, never the device memory: kernels get the
// address from scratch_device_address() instead.
static __device__ __align__(256) unsigned char scratch[kScratchBytes];

// Device address of each GPU's copy, looked up once per device (on the first call that
// needs it, with that device current) and kept.
constexpr int kScratchDevices = 64;
static std::mutex g_scratch_mu;
static void* g_scratch_addr[kScratchDevices];

hipError_t scratch_device_address(void** ptr) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kScratchDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_addr[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return e;
    if (!p) return hipErrorInvalidSymbol;
    g_scratch_addr[dev] = p;
  }
  *ptr = g_scratch_addr[dev];
  return hipSuccess;
}

// ---------------------------------------------------------------------------
// Launchers (host side).  Each returns the hipGetLastError() of its launch.
// Grid of a launch of n tiles with tail queues (sets tq.queue): the tiles plus the
// spare workgroups.
static unsigned queued_grid(int64_t n, TileQueue& tq) {
  const QueueShape qs = tq.ctr ? queue_shape(n) : QueueShape{0, 0};
  tq.queue = qs.queue;
  return (unsigned)(n + qs.spare);
}

hipError_t launch_fwd_tile(const FwdTileArgs& a, bool ent, hipStream_t s) {
  FwdTileArgs b = a;
  b.tq.clear = nullptr;
  const unsigned g = queued_grid((int64_t)a.n_mt * a.n_vt, b.tq);
  if (ent)
    fwd_tile_kernel<FwdShape, true><<<g, FwdShape::NTHREADS, 0, s>>>(b);
  else
    fwd_tile_kernel<FwdShape, false><<<g, FwdShape::NTHREADS, 0, s>>>(b);
  return hipGetLastError();
}

hipError_t launch_target_logit(const FwdTileArgs& a, hipStream_t s) {
  const unsigned g = (unsigned)(((long)a.M + TL_ROWS - 1) / TL_ROWS);
  target_logit_kernel<<<g, 64 * TL_ROWS, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_fwd_merge(const FwdMergeArgs& a, bool ent, hipStream_t s) {
  const unsigned g = (unsigned)((a.M + MERGE_ROWS - 1) / MERGE_ROWS);
  if (ent)
    fwd_merge_kernel<true><<<g, MERGE_ROWS * MERGE_SLICES, 0, s>>>(a);
  else
    fwd_merge_kernel<false><<<g, MERGE_ROWS * MERGE_SLICES, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_dlogits(const DlogitsArgs& a, bool entgrad, hipStream_t s) {
  DlogitsArgs b = a;
  const unsigned g = queued_grid((int64_t)a.n_mt * a.n_vt, b.tq);
  if (entgrad)
    bwd_dlogits_kernel<true><<<g, NTHREADS, 0, s>>>(b);
  else
    bwd_dlogits_kernel<false><<<g, NTHREADS, 0, s>>>(b);
  return hipGetLastError();
}

hipError_t launch_bwd_pipe(const PipeArgs& a, bool entgrad, hipStream_t s) {
  const long per = (a.n_dw + 7) / 8 + (a.n_dx + 7) / 8 + (a.n_dl + 7) / 8;
  if (per == 0) return hipSuccess;
  if (entgrad)
    bwd_pipe_kernel<true><<<(unsigned)(8 * per), NTHREADS, 0, s>>>(a);
  else
    bwd_pipe_kernel<false><<<(unsigned)(8 * per), NTHREADS, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_gemm_dw(const GemmDwArgs& a, hipStream_t s) {
  GemmDwArgs b = a;
  const unsigned g = queued_grid((int64_t)a.n_i * a.n_h, b.tq);
  gemm_dw_kernel<<<g, NTHREADS, 0, s>>>(b);
  return hipGetLastError();
}

hipError_t launch_gemm_dx(const GemmDxArgs& a, hipStream_t s) {
  gemm_dx_kernel<<<(unsigned)((long)a.n_m * a.n_h), NTHREADS, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_nll_reduce(const float* logprob, const int64_t* targets, long M, int64_t V,
                             int64_t ignore_index, double* out, hipStream_t s) {
  nll_reduce_kernel<<<1, NLL_THREADS, 0, s>>>(logprob, targets, M, V, ignore_index, out);
  return hipGetLastError();
}

hipError_t launch_nll_mean_grad(const int64_t* targets, long M, int64_t V, int64_t ignore_index,
                                const double* reduced, float* grad, hipStream_t s) {
  long blocks = (M + 255) / 256;
  if (blocks > 4096) blocks = 4096;
  nll_mean_grad_kernel<<<(unsigned)blocks, 256, 0, s>>>(targets, M, V, ignore_index, reduced, grad);
  return hipGetLastError();
}

hipError_t launch_policy_loss_reduce(const PolicyLossArgs& a, float* per_token_loss,
                                     uint8_t* is_clipped, double* out, hipStream_t s) {
  policy_loss_reduce_kernel<<<1, PL_THREADS, 0, s>>>(a, per_token_loss, is_clipped, out);
  return hipGetLastError();
}

hipError_t launch_policy_loss_grad(const PolicyLossArgs& a, const double* reduced, float* grad,
                                   hipStream_t s) {
  long blocks = (a.M + 255) / 256;
  if (blocks > 4096) blocks = 4096;
  policy_loss_grad_kernel<<<(unsigned)blocks, 256, 0, s>>>(a, reduced, grad);
  return hipGetLastError();
}

hipError_t launch_fill_zero_u16(uint16_t* p, long n, hipStream_t s) {
  if (n <= 0) return hipSuccess;
  long blocks = (n + 255) / 256;
  if (blocks > 65536) blocks = 65536;
  fill_u16_kernel<<<(unsigned)blocks, 256, 0, s>>>(p, n);
  return hipGetLastError();
}

}  // namespace flce
