// Device code shared by the tile kernels of libflce (gfx950): tile shapes, tile
// coordinates and tail queues, direct-to-LDS loads of operand tiles, and the epilogue
// that reduces a transposed logit tile to per-token softmax partials.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "flce_internal.h"

#define LDS_AS __attribute__((address_space(3)))

namespace flce {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int NTHREADS = 256;    // 4 waves of 64 in a 2 x 2 grid over the workgroup tile
// Pin the instruction order of a sub-step: the fragment reads of sub-step kk + 1
// alternate with the first MFMAs of sub-step kk, so each read is issued a whole
// sub-step before its first use.  Left to itself the scheduler reuses fragment
// registers right after their last MFMA and issues each read only one MFMA group
// ahead, exposing the LDS latency.
constexpr bool SCHED_PIPE = true;
// A stage's loads are issued in LOAD_GROUPS groups per MFMA sub-step (at most one
// group per MFMA), placed between the sub-step's MFMA groups: half of them under the
// last sub-step of the step before (right after the barrier that frees their stage),
// the others under sub-step 0.  Measured best: 16 groups and half early (8 groups
// tie; 4 or 12 early loads cost 1.5-3%).
constexpr int LOAD_GROUPS = 16;
constexpr uint32_t OOB_OFFSET = 0x80000000u;  // beyond every descriptor's num_records
constexpr uint32_t RSRC_WORD3 = 0x00020000u;  // raw buffer, 32-bit data format

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// Shape of a workgroup's mainloop: a TM x TN output tile computed by 4 waves of
// (TM / 2) x (TN / 2), K staged BK at a time through NST LDS stages.  WAVES_PER_EU
// is the occupancy the register budget is sized for: 2 lets two workgroups share a
// CU, so one workgroup's barrier and load-issue stalls hide under the other's
// matrix work (their LDS footprints must then fit 160 KiB together).
template <int TM_, int TN_, int BK_, int NST_, int WAVES_PER_EU_, int WAVES_M_ = 2,
          int WAVES_N_ = 2>
struct Shape {
  static constexpr int TM = TM_, TN = TN_, BK = BK_, NST = NST_;
  static constexpr int WAVES_PER_EU = WAVES_PER_EU_;
  static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;  // wave grid over the tile
  static constexpr int NWAVES = WAVES_M * WAVES_N, NTHREADS = 64 * NWAVES;
  static constexpr int WM = TM / WAVES_M, WN = TN / WAVES_N;    // wave tile
  static constexpr int MB = WM / 32, NB = WN / 32;    // 32 x 32 MFMA blocks per wave
  static constexpr int KK = BK / 16;                  // MFMA sub-steps per stage
  static constexpr int A_BYTES = TM * BK * 2, B_BYTES = TN * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int PIPE_BYTES = NST * STAGE_BYTES;
  static constexpr int DMA_A = A_BYTES / (1024 * NWAVES), DMA_B = B_BYTES / (1024 * NWAVES);  // 1 KiB loads per wave
  static constexpr int DMA_STAGE = DMA_A + DMA_B;
  static_assert(MB >= 2 && MB % 2 == 0 && NB >= 1, "wave tile");
  static_assert(BK == 32 || BK == 64, "K per stage");
  static_assert(A_BYTES % (1024 * NWAVES) == 0 && B_BYTES % (1024 * NWAVES) == 0,
                "whole loads per wave");
  static_assert(NST >= 2 && NST <= 4, "stages");
};
// One workgroup per CU: 256 x 256 tiles, waves of 128 x 128, 128 KiB of LDS stages.
using BigShape = Shape<256, 256, 64, 2, 1>;
// The forward runs BigShape.  Eight waves of 128 x 64 (two per SIMD, Shape<256, 256,
// 64, 2, 2, 2, 4>) hide more stalls but read 1.5x the LDS; with the lean K loop they
// measured 5% slower.
using FwdShape = BigShape;
static_assert(FwdShape::TM == kFwdTileM && FwdShape::TN == kFwdTileN, "host and kernel tile");
constexpr int FWD_GROUP_M = 2048 / kFwdTileM;  // forward tile rows per L2 group

// ---------------------------------------------------------------------------
// Tile coordinates.  Workgroups are handed to the 8 XCDs round robin, so id b runs
// on XCD b % 8.  Ids are renumbered so each XCD receives a contiguous range of
// logical ids, walked in groups of `group_m` tile rows (tile row fastest): the
// workgroups resident on one XCD then share a few operand tiles in its L2.
// Logical id L of a grid of n_m x n_n tiles -> tile (tm, tn): groups of `group_m` tile
// rows, tile row fastest within a group.
__device__ __forceinline__ void group_coords(int L, int n_m, int n_n, int group_m, int& tm,
                                             int& tn) {
  const int width = group_m * n_n;
  const int g = L / width;
  const int first = g * group_m;
  const int gm = min(n_m - first, group_m);
  const int inner = L - g * width;
  tm = first + inner % gm;
  tn = inner / gm;
}

__device__ __forceinline__ void tile_coords(int bid, int nblocks, int n_m, int n_n, int group_m,
                                            int& tm, int& tn) {
  const int per = nblocks >> 3;
  int L = bid;
  if (bid < (per << 3)) L = (bid & 7) * per + (bid >> 3);
  group_coords(L, n_m, n_n, group_m, tm, tn);
}

// Queued tiles left in a counter (negative once exhausted).
__device__ __forceinline__ long long queue_left(unsigned long long c, int q) {
  return (long long)q - (long long)(c & 0xffffffffull) - (long long)(c >> 32);
}

// Logical id of this workgroup's tile for a launch of n tiles plus spare workgroups,
// with the last tq.queue ids of each XCD's stream (the logical ids x * per ... of
// tile_coords) taken through the counters of TileQueue; -1 when the workgroup finds
// no tile.  Lane 0 of wave 0 claims: a workgroup of the stream first from the front of
// its own XCD's queue, then (a spare at once) from the back of the queue with the most
// tiles left, until every queue is empty (each pass either takes a tile or sees a
// counter that only grows, so the loop ends).
// The bounds on both counts keep every id in range whatever the counters hold.
// Workgroup 0 also zeroes tq.clear for a later launch.
__device__ __forceinline__ int tile_claim(int n, const TileQueue& tq) {
  const int bid = blockIdx.x;
  if (bid == 0 && threadIdx.x < 8 && tq.clear)
    __hip_atomic_store(&tq.clear[threadIdx.x], 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const int per = n >> 3, q = tq.queue, x = bid & 7;
  if (bid < (per << 3)) {
    if ((bid >> 3) < per - q) return x * per + (bid >> 3);
  } else if (bid < n) {
    return bid;
  }
  if (q == 0) return -1;
  __shared__ int claimed;
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    const unsigned long long uq = (unsigned long long)q;
    int L = -1;
    if (lane == 0 && bid < n) {
      const unsigned long long old = atomicAdd(&tq.ctr[x], 1ull);
      const unsigned long long f = old & 0xffffffffull, b = old >> 32;
      if (f < uq && b < uq - f) L = x * per + per - q + (int)f;
    }
    L = __shfl(L, 0);
    while (L < 0) {
      const long long left =
          lane < 8 ? queue_left(__hip_atomic_load(&tq.ctr[lane & 7], __ATOMIC_RELAXED,
                                                  __HIP_MEMORY_SCOPE_AGENT), q)
                   : 0;
      int y = -1;
      long long most = 0;
      for (int j = 0; j < 8; ++j) {
        const long long r = __shfl(left, j);
        if (r > most) {
          most = r;
          y = j;
        }
      }
      if (y < 0) break;
      if (lane == 0) {
        const unsigned long long old = atomicAdd(&tq.ctr[y], 1ull << 32);
        const unsigned long long f = old & 0xffffffffull, b = old >> 32;
        if (b < uq && f < uq - b) L = y * per + per - 1 - (int)b;
      }
      L = __shfl(L, 0);
    }
    if (lane == 0) claimed = L;
  }
  __syncthreads();
  return claimed;
}

// ---------------------------------------------------------------------------
// One operand of the mainloop, as seen by a workgroup.
//  K-contiguous (KC): `base` is element (row 0 of the tile, k = 0) of a [rows][K]
//     matrix with leading dimension ld; `valid` rows of the tile exist.
//  M/N-contiguous (MN): `base` is element (k = 0, column 0 of the tile) of a
//     [K][cols] matrix with leading dimension ld; `valid` columns of the tile exist.
// `kvalid` is the K extent that exists.  `band` = 0 for a row-major matrix; otherwise
// the matrix is tile-blocked (the d-logit buffer): 256-row bands of `band` elements,
// each a row of 256 x 64 blocks (16384 elements, row r of a block at 64 r).  A KC
// operand then reads the rows of its band (base = the band's start, ld = 64) and moves
// one block per 64 K; an MN operand reads 64-column blocks of consecutive K rows
// (base = block 0 of band 0 of its columns).
constexpr int BLK_ROWS = 256, BLK_COLS = 64, BLK_ELEMS = BLK_ROWS * BLK_COLS;
static_assert(BigShape::BK == BLK_COLS && BigShape::TM == BLK_ROWS, "one block per K step");
struct TileSrc {
  const uint16_t* base;
  long ld;
  int valid;
  int kvalid;
  long band;
};

// LDS layout of a KC tile: rows of BK bf16 (BK / 8 chunks of 16 bytes); chunk c of
// row r sits at chunk position c ^ kc_swz(r).  The 16 rows one ds_read_b128 cycle
// serves land on 16 distinct 16-byte bank groups.
template <int CHUNKS>
__device__ __forceinline__ int kc_swz(int r) {
  return CHUNKS == 8 ? ((r ^ (r >> 3)) & 7) : ((r >> 2) & 3);
}

// LDS layout of an MN tile of `cols` columns: BK K rows of 2 cols bytes (cols / 16
// blocks of 32 bytes); block b of K row k sits at block position b ^ mn_swz(k).  Each
// half-wave of a transposing fragment read takes two adjacent blocks (2j, 2j + 1) of
// 4 consecutive K rows; mn_swz maps those 4 rows to {0, 2, 5, 7}, so the 8 (row,
// block) pairs fall on the 8 distinct 32-byte bank groups of the 256-byte bank row
// (with k & 7 as the swizzle they took only 4, a 2-way conflict on every read).
__device__ __forceinline__ int mn_swz(int k) { return ((k & 3) << 1) ^ ((k >> 1) & 1); }

// One 64-lane direct-to-LDS load: lane i's 16 bytes from byte offset voff of the
// buffer go to LDS address lds_addr + 16 i.  Issued as inline assembly so that the
// compiler does not treat the fragment reads of the other stages as dependent on
// it; the mainloop waits for these loads itself (s_waitcnt vmcnt) before the
// barrier that publishes a stage.
typedef int i32x4 __attribute__((ext_vector_type(4)));
template <int IMM>
__device__ __forceinline__ void dma16(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds_addr) {
  static_assert(IMM >= 0 && IMM < 4096, "buffer instruction offset range");
  asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dwordx4 %0, %1, %2 offen offset:%4 lds"
               :
               : "v"(voff), "s"(rsrc), "s"(soff), "s"(lds_addr), "i"(IMM)
               : "memory");
}

// The same without rewriting m0: the LDS destination is the m0 of the previous
// dma16 plus IMM (the immediate offset applies to the LDS address as well as to the
// global one, which the lane offsets pre-subtract).
template <int IMM>
__device__ __forceinline__ void dma16_same_m0(i32x4 rsrc, uint32_t voff, uint32_t soff) {
  static_assert(IMM >= 0 && IMM < 4096, "buffer instruction offset range");
  asm volatile("buffer_load_dwordx4 %0, %1, %2 offen offset:%3 lds"
               :
               : "v"(voff), "s"(rsrc), "s"(soff), "i"(IMM)
               : "memory");
}

// Buffer descriptor with a fixed record count: every lane that must not load
// already carries an offset >= OOB_OFFSET, which the buffer unit turns into zeros.
__device__ __forceinline__ i32x4 make_rsrc_fixed(const void* base) {
  const unsigned long a = (unsigned long)base;
  i32x4 r;
  r.x = __builtin_amdgcn_readfirstlane((int)(a & 0xffffffffu));
  r.y = __builtin_amdgcn_readfirstlane((int)((a >> 32) & 0xffffu));
  r.z = 0x7fffffff;
  r.w = (int)RSRC_WORD3;
  return r;
}

__device__ __forceinline__ uint32_t lds_addr_of(const char* p) {
  return (uint32_t)(uintptr_t)(LDS_AS const char*)p;
}

// Direct-to-LDS loads of one ROWS x BK operand tile (ROWS rows of a KC operand, or
// ROWS columns of an MN operand).  The tile is filled by 4 waves x N loads; load j
// of wave w fills LDS bytes [(w N + j) KiB, + 1 KiB) of the tile, lane i the 16
// bytes at i * 16.  Each lane's byte offsets relative to the K step's base address
// do not change from step to step, so they are computed once, together with the K
// position of the lane's 16 bytes within the step (in 8-element chunks for KC, in
// K rows for MN, one byte per load).  A step keeps the loads whose K position lies
// below a uniform limit and turns the others into zero fills, without branches.
template <bool KC, int ROWS, int BK, int NWAVES = 4>
struct DmaPlan {
  static constexpr int N = ROWS * BK * 2 / (1024 * NWAVES);  // loads per wave
  static constexpr int CHUNKS = BK / 8;           // KC: 16-byte chunks per tile row
  static constexpr int GPR = ROWS / 8;            // MN: 16-byte granules per K row
  static constexpr int KPOS_MAX = KC ? CHUNKS : BK;
  uint32_t voff[N];
  int wave;
  i32x4 rsrc0;         // buffer descriptor of the tile's base (k = 0), wave-uniform
  uint32_t kc_bytes;   // KC: bytes per K element (2, or 512 in a blocked matrix)
  uint32_t row_bytes;  // MN: bytes per K row within a 256-row band
  uint32_t band_bytes; // MN: bytes per 256-row band

  __device__ __forceinline__ void init(const TileSrc& s, int wave_id) {
    wave = wave_id;
    rsrc0 = make_rsrc_fixed(s.base);
    const bool blk = s.band != 0;
    kc_bytes = blk ? 2u * BLK_ROWS : 2u;
    row_bytes = (uint32_t)__builtin_amdgcn_readfirstlane((int)(blk ? 2 * BLK_COLS : s.ld * 2));
    band_bytes = (uint32_t)__builtin_amdgcn_readfirstlane(
        (int)(blk ? s.band * 2 : (long)BLK_ROWS * s.ld * 2));
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int G = (wave * N + j) * 64 + lane;  // 16-byte granule of the tile
      int a, b;
      if constexpr (KC) {
        a = G / CHUNKS;                          // tile row
        b = (G % CHUNKS) ^ kc_swz<CHUNKS>(a);    // 16-byte chunk of K in the row
      } else {
        a = G / GPR;                             // K row
        b = (G % GPR) ^ (mn_swz(a) << 1);        // 16-byte chunk of columns
      }
      const bool ok = KC ? a < s.valid : 8 * b < s.valid;
      // element offset in the step: a blocked MN row's 16-byte chunk b lies in block b / 8
      const long e = (!KC && blk) ? (long)(b >> 3) * BLK_ELEMS + (long)a * BLK_COLS + 8 * (b & 7)
                                  : (long)a * s.ld + 8 * b;
      // the load's immediate offset (1 KiB x (j % 4)) is added back by the hardware
      voff[j] = (ok ? (uint32_t)(e * 2) : OOB_OFFSET) - 1024u * (j & 3);
    }
  }

  // K position of load j's 16 bytes within a step (a 16-byte chunk of K for KC, a K row
  // for MN), recomputed rather than kept: it is needed only in the few steps that
  // reach past K, and registers live across the K loop are the scarcest
  __device__ __forceinline__ int kpos(int j) const {
    const int G = (wave * N + j) * 64 + (int)(threadIdx.x & 63);
    if constexpr (KC) {
      const int a = G / CHUNKS;
      return (G % CHUNKS) ^ kc_swz<CHUNKS>(a);
    } else {
      return G / GPR;
    }
  }

  // offset of load j in a step of which `lim` K positions exist
  __device__ __forceinline__ uint32_t off(int j, int lim) const {
    return kpos(j) < lim ? voff[j] : OOB_OFFSET - 1024u * (j & 3);
  }
};

// Per-step state of one operand's loads.  A K-contiguous tile keeps one buffer base
// for the whole K loop and moves with the scalar offset (k0 times 2 bytes, or 512 in a
// blocked matrix, stays below 2^31); an M/N-contiguous tile moves its base by k0 rows
// (k0 / 256 bands and k0 % 256 rows of a band).  `lim` (uniform) is the
// number of the step's K positions that exist: 0 for a step past the end of K, whose
// loads then only zero-fill a free stage.
struct TileDma {
  i32x4 rsrc;
  uint32_t soff;
  uint32_t lds0;  // LDS byte address of this wave's first 1 KiB block of the tile
  int lim;
};

// FAST: the step lies entirely inside K (no per-lane K check, `lim` unused).  The
// descriptor and offsets are derived from the plan with scalar arithmetic only.
template <bool FAST, bool KC, int ROWS, int BK, int NW>
__device__ __forceinline__ TileDma tile_dma(const TileSrc& s, const DmaPlan<KC, ROWS, BK, NW>& plan,
                                            int k0, bool active, const char* lds_tile) {
  TileDma d;
  d.rsrc = plan.rsrc0;
  if constexpr (KC) {
    d.soff = (uint32_t)k0 * plan.kc_bytes;
  } else {
    const uint64_t base = ((uint64_t)(uint32_t)plan.rsrc0.y << 32 | (uint32_t)plan.rsrc0.x) +
                          (uint64_t)(uint32_t)(k0 >> 8) * plan.band_bytes +
                          (uint64_t)(uint32_t)(k0 & 255) * plan.row_bytes;
    d.rsrc.x = (int)(uint32_t)base;
    d.rsrc.y = (int)((base >> 32) & 0xffffu);
    d.soff = 0u;
  }
  d.lds0 = lds_addr_of(lds_tile) + (uint32_t)(plan.wave * plan.N * 1024);
  if constexpr (FAST) {
    d.lim = KC ? plan.CHUNKS : BK;
  } else {
    const int rem = s.kvalid - k0;  // K extent left from k0 (a multiple of 8 for KC)
    d.lim = !active ? 0 : KC ? min(max((rem + 7) >> 3, 0), plan.CHUNKS) : min(max(rem, 0), BK);
  }
  return d;
}

// Load j of a tile.  m0 holds the LDS base of a group of 4 loads; `set_m0` rewrites
// it (required for the first load issued after any other code that may touch m0 is
// scheduled in between), the other loads of the group ride on the immediate offset.
template <bool FAST, bool KC, int ROWS, int BK, int NW>
__device__ __forceinline__ void tile_load(const TileDma& d, const DmaPlan<KC, ROWS, BK, NW>& plan, int j,
                                          bool set_m0) {
  const uint32_t v = FAST ? plan.voff[j] : plan.off(j, d.lim);
  const uint32_t m0 = d.lds0 + (uint32_t)(j & ~3) * 1024u;
  switch (j & 3) {
    case 0: dma16<0>(d.rsrc, v, d.soff, m0); break;
    case 1: if (set_m0) dma16<1024>(d.rsrc, v, d.soff, m0); else dma16_same_m0<1024>(d.rsrc, v, d.soff); break;
    case 2: if (set_m0) dma16<2048>(d.rsrc, v, d.soff, m0); else dma16_same_m0<2048>(d.rsrc, v, d.soff); break;
    default: if (set_m0) dma16<3072>(d.rsrc, v, d.soff, m0); else dma16_same_m0<3072>(d.rsrc, v, d.soff); break;
  }
}

// The loads of one whole stage: stage load j < DMA_A is load j of the A tile, the
// rest are the B tile's (B_FIRST: the other way round).  The first half of a stage's
// loads goes out early (right after a barrier), so the order decides which operand
// waits longer: issuing the L2-resident operand first measured faster (forward with W
// first: +3%; dW with X^T first: -0.4%; dX with W first: +0.3%).
template <class S, bool A_KC, bool B_KC, bool FAST = false, bool B_FIRST = false>
struct StageDma {
  using PA = DmaPlan<A_KC, S::TM, S::BK, S::NWAVES>;
  using PB = DmaPlan<B_KC, S::TN, S::BK, S::NWAVES>;
  TileDma a, b;
  const PA* pa;
  const PB* pb;
  // issue stage loads [j0, j1) back to back (B_FIRST: the B tile's loads come first)
  __device__ __forceinline__ void issue(int j0, int j1) const {
    constexpr int DF = B_FIRST ? S::DMA_B : S::DMA_A;  // loads of the first tile
#pragma unroll
    for (int j = j0; j < j1; ++j) {
      if (j < DF) {
        if constexpr (B_FIRST) tile_load<FAST>(b, *pb, j, j == j0);
        else tile_load<FAST>(a, *pa, j, j == j0);
      } else {
        if constexpr (B_FIRST) tile_load<FAST>(a, *pa, j - DF, j == j0 || j == DF);
        else tile_load<FAST>(b, *pb, j - DF, j == j0 || j == DF);
      }
    }
  }
};

// s_waitcnt until at most n of this wave's vector-memory operations are outstanding
// (expcnt and lgkmcnt left unconstrained).
template <int n>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14));
}
// Row of the wave tile held by lane `lane` in element e of a 32 x 32 block.
__device__ __forceinline__ int acc_row(int lane, int e) {
  return ((e >> 2) << 3) + ((lane >> 5) << 2) + (e & 3);
}

// v_max_f32 without the quieting of its inputs that fmaxf adds (the inputs are MFMA
// results or maxima of them, never signaling NaNs).
__device__ __forceinline__ float max_raw(float a, float b) {
  float r;
  asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

// v_permlane32_swap_b32: the upper half-wave of a (lanes 32-63) trades places with the
// lower half-wave of b, so that afterwards a holds (own a | b of lane - 32) and b holds
// (a of lane + 32 | own b).  Issued as inline assembly because the compiler builtin
// hands back only the first register; the s_nop pads cover the VALU hazards around it.
__device__ __forceinline__ void swap32(float& a, float& b) {
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1\n\ts_nop 1" : "+v"(a), "+v"(b));
}

// x and y each combined over lanes l and l ^ 32 in one swap: the result is that of x
// in the lower half-wave and that of y in the upper one.
template <class Op>
__device__ __forceinline__ float halves_reduce(float x, float y, Op op) {
  swap32(x, y);
  return op(x, y);
}

// A value bounded by 0 from above or from below.  By comparison, so that a NaN stays one:
// fminf and fmaxf hand back the operand that is a number.
__device__ __forceinline__ float at_most_zero(float v) { return v > 0.f ? 0.f : v; }
__device__ __forceinline__ float at_least_zero(float v) { return v < 0.f ? 0.f : v; }

// log of a row's sum of shifted exponentials.  The largest term is 2^r, r being what rounding
// took from the shift (half a step of the largest logit in log2 units): 64 at logits of 2^30.  Of
// logits twice as large and more the sum can come out 0 or infinite, which says nothing about
// the row: NaN.
__device__ __forceinline__ float log_sum(float s) {
  return s > 0.f && s < INFINITY ? logf(s) : __uint_as_float(0x7fc00000u);
}

// max(m, sgn a, sgn b) with sgn = -1 under NEG, as one v_max3_f32 issued directly:
// fmaxf on values the compiler cannot prove to be quiet NaNs (here, MFMA results)
// costs one quieting v_max per input.  m is already a running maximum of sgn-scaled
// values, so only a and b take the negation modifier.
template <bool NEG>
__device__ __forceinline__ float max3_run(float m, float a, float b) {
  float r;
  if constexpr (NEG)
    asm("v_max3_f32 %0, %1, -%2, -%3" : "=v"(r) : "v"(m), "v"(a), "v"(b));
  else
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(m), "v"(a), "v"(b));
  return r;
}

// Per token column of the lane, the maximum of sgn * acc over the lane's 16 MB
// vocabulary rows (sgn = -1 if NEG; the maximum of z = scale * acc is |scale| times
// that of sgn(scale) * acc); rows at or past `vrows` of the wave tile are skipped when
// RAGGED.
template <bool NEG, bool RAGGED, class S>
__device__ __forceinline__ void lane_col_max(const f32x16 (&acc)[S::MB][S::NB], int lane,
                                             int vrows, float (&mx)[S::NB]) {
  constexpr float SKIP = NEG ? INFINITY : -INFINITY;  // what the maximum ignores
#pragma unroll
  for (int nb = 0; nb < S::NB; ++nb) mx[nb] = -INFINITY;
#pragma unroll
  for (int mb = 0; mb < S::MB; ++mb)
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const bool v0 = !RAGGED || 32 * mb + acc_row(lane, e) < vrows;
      const bool v1 = !RAGGED || 32 * mb + acc_row(lane, e + 1) < vrows;
#pragma unroll
      for (int nb = 0; nb < S::NB; ++nb)
        mx[nb] = max3_run<NEG>(mx[nb], v0 ? acc[mb][nb][e] : SKIP, v1 ? acc[mb][nb][e + 1] : SKIP);
    }
}

// Per token column of the lane, the shifted sums over its 16 MB vocabulary rows in
// log2 units: s = sum 2^d and u = sum 2^d d with d = c1 z - m2 (nm2 = -m2 per column).
template <bool ENT, bool RAGGED, class S>
__device__ __forceinline__ void lane_col_sums(const f32x16 (&acc)[S::MB][S::NB], int lane,
                                              int vrows, float c1, const float (&nm2)[S::NB],
                                              float (&sv)[S::NB], float (&uv)[S::NB]) {
#pragma unroll
  for (int nb = 0; nb < S::NB; ++nb) sv[nb] = uv[nb] = 0.f;
#pragma unroll
  for (int mb = 0; mb < S::MB; ++mb)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const bool valid = !RAGGED || 32 * mb + acc_row(lane, e) < vrows;
#pragma unroll
      for (int nb = 0; nb < S::NB; ++nb) {
        float d = fmaf(acc[mb][nb][e], c1, nm2[nb]);
        if constexpr (RAGGED) d = valid ? d : -INFINITY;
        const float pe = __builtin_amdgcn_exp2f(d);
        sv[nb] += pe;
        if constexpr (ENT) uv[nb] = fmaf(pe, RAGGED ? fmaxf(d, -3.0e38f) : d, uv[nb]);
      }
    }
}

// Epilogue of a forward tile of TN tokens x TM vocabulary entries of the logits, computed
// transposed: z^T = W X^T, the MFMA rows being vocabulary entries and its columns
// tokens.  Per wave, lane l then holds, for each of its NB token columns 32 nb + l % 32,
// 16 MB vocabulary rows of the wave tile, so the maxima and sums over the vocabulary
// run down the lane's own registers, meet the other half-wave in one swap, and meet the
// other wave of the same tokens through LDS.  The maximum over the tile's TM entries is
// formed first, so both row halves sum against the same shift and their partials simply
// add; thread t < TN writes the partials of token t of the tile.
template <class S, bool ENT>
__device__ __forceinline__ void fwd_epilogue(const f32x16 (&acc)[S::MB][S::NB], char* smem,
                                             const FwdTileArgs& p, int mt, int vt) {
  constexpr int TV = S::TM, TT = S::TN, NB = S::NB, WM = S::WM, WN = S::WN;
  constexpr int RP = S::WAVES_M;  // row parts: waves sharing the same tokens
  static_assert(NB % 2 == 0, "token columns pair up across the half-waves");
  static_assert(3 * RP * TT * 4 <= S::PIPE_BYTES, "epilogue buffers");
  const int row0 = mt * TT, col0 = vt * TV;  // first token, first vocabulary entry
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // wave-uniform

  const int wm = wave / S::WAVES_N;
  const int wv0 = wm * WM, wt0 = (wave % S::WAVES_N) * WN;
  const int lc = lane & 31, hi = lane >> 5;
  const float c1 = p.scale * LOG2E;  // logits in log2 units: z2 = c1 acc
  const float ac1 = fabsf(c1);
  const bool ragged = col0 + TV > p.V;
  const int vrows = p.V - col0 - wv0;  // vocabulary rows of the wave tile that exist

  // epilogue LDS: token maxima per row part [RP][TT], sums [RP][2][TT]
  float* red = reinterpret_cast<float*>(smem);
  float* comb = red + RP * TT;

  // maxima of sgn(c1) z over the wave's vocabulary rows: lane, then half-wave (token
  // columns 2 j + hi of the lane come out in half hi), then the row parts via LDS
  {
    float mx[NB];
    if (!ragged) {
      if (c1 >= 0.f) lane_col_max<false, false, S>(acc, lane, vrows, mx);
      else lane_col_max<true, false, S>(acc, lane, vrows, mx);
    } else {
      if (c1 >= 0.f) lane_col_max<false, true, S>(acc, lane, vrows, mx);
      else lane_col_max<true, true, S>(acc, lane, vrows, mx);
    }
#pragma unroll
    for (int j = 0; j < NB / 2; ++j)
      red[wm * TT + wt0 + 32 * (2 * j + hi) + lc] =
          halves_reduce(mx[2 * j], mx[2 * j + 1], [](float a, float b) { return max_raw(a, b); });
  }
  __syncthreads();

  // shifted sums against the tile maximum of each token column
  {
    float nm2[NB], sv[NB], uv[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float m = red[wt0 + 32 * nb + lc];
#pragma unroll
      for (int rp = 1; rp < RP; ++rp) m = fmaxf(m, red[rp * TT + wt0 + 32 * nb + lc]);
      nm2[nb] = -ac1 * m;
    }
    if (!ragged)
      lane_col_sums<ENT, false, S>(acc, lane, vrows, c1, nm2, sv, uv);
    else
      lane_col_sums<ENT, true, S>(acc, lane, vrows, c1, nm2, sv, uv);
#pragma unroll
    for (int j = 0; j < NB / 2; ++j) {
      const int t = wt0 + 32 * (2 * j + hi) + lc;
      comb[(2 * wm) * TT + t] =
          halves_reduce(sv[2 * j], sv[2 * j + 1], [](float a, float b) { return a + b; });
      if constexpr (ENT)
        comb[(2 * wm + 1) * TT + t] =
            halves_reduce(uv[2 * j], uv[2 * j + 1], [](float a, float b) { return a + b; });
    }
  }
  __syncthreads();
  if (tid < TT) {
    float mx = red[tid], sm = comb[tid], um = comb[TT + tid];
#pragma unroll
    for (int rp = 1; rp < RP; ++rp) {
      mx = fmaxf(mx, red[rp * TT + tid]);
      sm += comb[(2 * rp) * TT + tid];
      if constexpr (ENT) um += comb[(2 * rp + 1) * TT + tid];
    }
    const long off = (long)vt * p.Mpad + row0 + tid;
    p.part_m[off] = ac1 * mx * LN2;
    p.part_s[off] = sm;
    if constexpr (ENT) p.part_u[off] = um * LN2;
  }
}

}  // namespace flce
