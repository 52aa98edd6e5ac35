// The bf16 MFMA mainloop shared by the tile kernels of libflce (gfx950): fragments of operands
// in either memory order, the software pipeline over K, and reads of the accumulators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "tile_device.h"

namespace flce {

// Per-lane LDS byte offsets of the MFMA fragments a wave reads from one operand
// tile, for sub-step kk = 0; sub-step kk adds a constant (folded into the LDS
// instruction's immediate offset where the layout allows).
//  KC tile: fragment of rows idx0 + lane % 32, K chunk 2 kk + lane / 32 (ds_read_b128).
//  MN tile: the same fragment with two transposing reads; in each 16-lane group,
//  lane i reads 4 columns (4 (i % 4) .. + 3 of the group's 16) of K row i / 4 and
//  the read hands lane j of the group column j of those 4 K rows.
template <bool KC, int NBLK, int ROWS, int BK>
struct FragPlan {
  static constexpr int ROW_BYTES = KC ? BK * 2 : ROWS * 2;  // bytes per LDS row
  uint32_t off[NBLK][KC ? BK / 16 : 2];  // [block][kk] for KC, [block][half] for MN

  // region: LDS byte offset of the operand's stage-0 tile, folded into the offsets so
  // that a stage is selected by an instruction's immediate offset
  __device__ __forceinline__ void init(int idx_base, int lane, uint32_t region) {
#pragma unroll
    for (int blk = 0; blk < NBLK; ++blk) {
      const int idx0 = idx_base + 32 * blk;
      if constexpr (KC) {
        const int r = idx0 + (lane & 31);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
          const int c = 2 * kk + (lane >> 5);
          off[blk][kk] = region + r * ROW_BYTES + ((c ^ kc_swz<BK / 8>(r)) << 4);
        }
      } else {
        const int g = lane >> 4, i = lane & 15;
        const int c0 = idx0 + 16 * (g & 1) + 4 * (i & 3);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int k = 8 * (g >> 1) + 4 * hh + (i >> 2);  // kk adds 16 rows: mn_swz unchanged
          off[blk][hh] = region + k * ROW_BYTES + (((c0 >> 4) ^ mn_swz(k)) << 5) + ((c0 & 15) << 1);
        }
      }
    }
  }

  __device__ __forceinline__ bf16x8 read(const char* tile, int blk, int kk) const {
    if constexpr (KC) {
      return *reinterpret_cast<const bf16x8*>(tile + off[blk][kk]);
    } else {
      const i16x4 h0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (LDS_AS i16x4*)(tile + off[blk][0] + kk * 16 * ROW_BYTES));
      const i16x4 h1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (LDS_AS i16x4*)(tile + off[blk][1] + kk * 16 * ROW_BYTES));
      const i16x8 v = {h0[0], h0[1], h0[2], h0[3], h1[0], h1[1], h1[2], h1[3]};
      return __builtin_bit_cast(bf16x8, v);
    }
  }
};

template <class S, bool A_KC, bool B_KC>
struct Frags {
  FragPlan<A_KC, S::MB, S::TM, S::BK> a;
  FragPlan<B_KC, S::NB, S::TN, S::BK> b;
};

// The LDS tiles of one K step: A and B operand tiles.
struct StagePtr {
  const char* a;
  const char* b;
};

template <class S, bool A_KC, bool B_KC>
__device__ __forceinline__ void read_frags(bf16x8 (&af)[S::MB], bf16x8 (&bfr)[S::NB],
                                           StagePtr stage, const Frags<S, A_KC, B_KC>& f, int kk) {
#pragma unroll
  for (int mb = 0; mb < S::MB; ++mb) af[mb] = f.a.read(stage.a, mb, kk);
#pragma unroll
  for (int nb = 0; nb < S::NB; ++nb) bfr[nb] = f.b.read(stage.b, nb, kk);
}

template <int MB, int NB>
__device__ __forceinline__ void mfma_block(f32x16 (&acc)[MB][NB], const bf16x8 (&af)[MB],
                                           const bf16x8 (&bfr)[NB]) {
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      acc[mb][nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[mb], bfr[nb], acc[mb][nb], 0, 0, 0);
}


// Fragment i of sub-step kk: i < MB is A block i, the others B block i - MB.
template <class S, bool A_KC, bool B_KC>
__device__ __forceinline__ void read_frag(bf16x8 (&af)[S::MB], bf16x8 (&bfr)[S::NB],
                                          StagePtr stage, const Frags<S, A_KC, B_KC>& f, int kk,
                                          int i) {
  if (i < S::MB)
    af[i] = f.a.read(stage.a, i, kk);
  else
    bfr[i - S::MB] = f.b.read(stage.b, i - S::MB, kk);
}

// LDS read instructions of fragments [i0, i1) (a transposing fragment takes two).
template <class S, bool A_KC, bool B_KC>
constexpr int frag_read_instrs(int i0, int i1) {
  int n = 0;
  for (int i = i0; i < i1; ++i) n += (i < S::MB ? A_KC : B_KC) ? 1 : 2;
  return n;
}

// Group g (of GROUPS) of one MFMA sub-step: a share of the fragment reads of
// sub-step RKK of the stage at `rstage` (the next sub-step), each paired with one
// of the group's MFMAs, the group's other MFMAs, then a share of the stage loads
// [JB, JE) of `dma`.  Scheduling fences keep the loads between the MFMA groups, so
// the matrix pipe never waits behind a long burst of load issue.
template <int RKK, int g, int GROUPS, int JB, int JE, class S, bool A_KC, bool B_KC, class Ops>
__device__ __forceinline__ void substep_group(f32x16 (&acc)[S::MB][S::NB],
                                              const bf16x8 (&af)[S::MB], const bf16x8 (&bfr)[S::NB],
                                              bf16x8 (&af_n)[S::MB], bf16x8 (&bfr_n)[S::NB],
                                              StagePtr rstage, const Frags<S, A_KC, B_KC>& f,
                                              Ops& dma) {
  constexpr int NF = S::MB + S::NB, F = S::MB * S::NB, D = JE - JB;
  constexpr int i0 = g * NF / GROUPS, i1 = (g + 1) * NF / GROUPS;
  constexpr int m0 = g * F / GROUPS, m1 = (g + 1) * F / GROUPS;
  constexpr int R = frag_read_instrs<S, A_KC, B_KC>(i0, i1);
  constexpr int P = R < m1 - m0 ? R : m1 - m0;
#pragma unroll
  for (int i = i0; i < i1; ++i) read_frag<S>(af_n, bfr_n, rstage, f, RKK, i);
#pragma unroll
  for (int m = m0; m < m1; ++m) {
    const int mb = m / S::NB, nb = m % S::NB;
    acc[mb][nb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[mb], bfr[nb], acc[mb][nb], 0, 0, 0);
  }
  if constexpr (SCHED_PIPE) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    if constexpr (m1 - m0 > P) __builtin_amdgcn_sched_group_barrier(0x008, m1 - m0 - P, 0);
    if constexpr (R > P) __builtin_amdgcn_sched_group_barrier(0x100, R - P, 0);
  }
  if constexpr (D > 0) {
    __builtin_amdgcn_sched_barrier(0);
    dma.issue(JB + g * D / GROUPS, JB + (g + 1) * D / GROUPS);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Sub-step kk (MFMAs on register set kk % 2) with the reads of sub-step RKK of
// `rstage` into the other set and stage loads [JB, JE) spread over GROUPS groups.
template <int kk, int RKK, int GROUPS, int JB, int JE, class S, bool A_KC, bool B_KC, class Ops,
          int... G>
__device__ __forceinline__ void substep_with_loads(f32x16 (&acc)[S::MB][S::NB],
                                                   bf16x8 (&af)[2][S::MB], bf16x8 (&bfr)[2][S::NB],
                                                   StagePtr rstage, const Frags<S, A_KC, B_KC>& f,
                                                   Ops& dma,
                                                   std::integer_sequence<int, G...>) {
  (substep_group<RKK, G, GROUPS, JB, JE, S>(acc, af[kk & 1], bfr[kk & 1], af[(kk + 1) & 1],
                                            bfr[(kk + 1) & 1], rstage, f, dma), ...);
}

// Pin the instruction order of one MFMA sub-step whose successor's fragments are
// read during it: (ds_read, MFMA) x P, then the remaining MFMAs or reads.  A
// transposing fragment takes two read instructions, so an M/N-contiguous operand
// doubles its share of the reads; left unpinned, the scheduler put the extra reads
// right before the MFMAs that use them, which then waited for all LDS reads.
template <class S, bool A_KC, bool B_KC, bool READS>
__device__ __forceinline__ void sched_substep() {
  constexpr int F = S::MB * S::NB;                                    // MFMAs per sub-step
  constexpr int R = frag_read_instrs<S, A_KC, B_KC>(0, S::MB + S::NB);  // read instructions
  constexpr int P = R < F ? R : F;                                    // reads paired with MFMAs
  if constexpr (SCHED_PIPE) {
    if constexpr (READS) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
      if constexpr (F > P) __builtin_amdgcn_sched_group_barrier(0x008, F - P, 0);
      if constexpr (R > P) __builtin_amdgcn_sched_group_barrier(0x100, R - P, 0);
    } else {
      __builtin_amdgcn_sched_group_barrier(0x008, F, 0);
    }
  }
}

// The MFMA mainloop shared by every kernel: D = A B^T over K for the workgroup's
// TM x TN tile, as 4 waves of WM x WN (wave w at rows WM (w / 2), columns
// WN (w % 2)).  acc[mb][nb] is the 32 x 32 block at (32 mb, 32 nb) of the wave
// tile in the v_mfma_f32_32x32x16 layout: lane l, element e holds row
// 8 (e / 4) + 4 (l / 32) + e % 4 and column l % 32.
//
// Pipeline: two LDS stages, laid out as A0, A1, B0, B1 (the B region's base is folded
// into the B fragment offsets, so every fragment read selects its stage with the
// instruction's immediate offset and the K loop, unrolled by two, issues no address
// arithmetic).  The KK MFMA sub-steps of stage kt run with the fragments of sub-step
// kk + 1 read (into the other register set) while the MFMAs of sub-step kk are
// issued.  Before the last sub-step the wave waits for its own loads of step kt + 1
// and the barrier publishes that stage and releases stage kt (all of whose reads
// have returned); the first fragments of step kt + 1 are then read under the last
// sub-step's MFMAs, so no step starts with an LDS-latency bubble.  The loads of step
// kt + 2 go out in groups between MFMA groups: the first EARLY of them under the last
// sub-step of step kt, right after the barrier freed their stage, the rest under
// sub-step 0 of step kt + 1.  Steps that lie entirely inside K take precomputed load
// offsets; the last steps check each lane's K position, and steps past K only
// zero-fill their stage, so every step issues the same number of loads and the wait
// before each barrier is a fixed count.  Steps run in pairs (stage 0, stage 1); an
// odd step count gets one step over a zero-filled stage.
template <class S, bool A_KC, bool B_KC, bool B_FIRST = false>
__device__ __forceinline__ void mainloop(f32x16 (&acc)[S::MB][S::NB], char* smem,
                                         const TileSrc& A, const TileSrc& B, int K) {
  static_assert(S::NST == 2, "two LDS stages");
  constexpr int KK = S::KK, D = S::DMA_STAGE;
  constexpr int EARLY = D / 2;
  constexpr int F = S::MB * S::NB, GR = LOAD_GROUPS < F ? LOAD_GROUPS : F;
  static_assert(EARLY > 0 && EARLY < 64, "early loads");
  static_assert(KK % 2 == 0, "sub-step 0 of every stage uses register set 0");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wr0 = (wave / S::WAVES_N) * S::WM, wc0 = (wave % S::WAVES_N) * S::WN;
#pragma unroll
  for (int mb = 0; mb < S::MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < S::NB; ++nb)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[mb][nb][e] = 0.f;

  const int nk = (K + S::BK - 1) / S::BK;
  // steps whose K range exists in both operands (an operand may hold fewer K rows than
  // the loop runs over, e.g. X's M rows against a K of M rounded up to 256)
  const int nfull = min(K, min(A.kvalid, B.kvalid)) / S::BK;
  typename StageDma<S, A_KC, B_KC>::PA plan_a;
  typename StageDma<S, A_KC, B_KC>::PB plan_b;
  const int wave_u = __builtin_amdgcn_readfirstlane(wave);
  plan_a.init(A, wave_u);
  plan_b.init(B, wave_u);
  Frags<S, A_KC, B_KC> frags;
  frags.a.init(wr0, lane, 0u);
  frags.b.init(wc0, lane, 2u * S::A_BYTES);
  // loads of step st into stage s; a step past K only zero-fills it
  auto stage_dma = [&](auto fast, int st, int s) {
    constexpr bool FAST = decltype(fast)::value;
    StageDma<S, A_KC, B_KC, FAST, B_FIRST> d;
    d.pa = &plan_a;
    d.pb = &plan_b;
    const bool active = st < nk;
    const int k0 = (active ? st : 0) * S::BK;
    d.a = tile_dma<FAST>(A, plan_a, k0, active, smem + s * S::A_BYTES);
    d.b = tile_dma<FAST>(B, plan_b, k0, active, smem + 2 * S::A_BYTES + s * S::B_BYTES);
    return d;
  };
  using Slow = std::integral_constant<bool, false>;
  using Fast = std::integral_constant<bool, true>;
  using Stage0 = std::integral_constant<int, 0>;
  using Stage1 = std::integral_constant<int, 1>;
  // prologue: step 0, and the early loads of step 1
  stage_dma(Slow(), 0, 0).issue(0, D);
  stage_dma(Slow(), 1, 1).issue(0, EARLY);
  wait_vmcnt<EARLY>();  // step 0 has landed
  __syncthreads();
  bf16x8 af[2][S::MB], bfr[2][S::NB];
  read_frags<S>(af[0], bfr[0], StagePtr{smem, smem}, frags, 0);
  constexpr auto groups = std::make_integer_sequence<int, GR>();
  // one K step computed from stage STG (kt % 2 == STG)
  auto step = [&](auto stg, auto fast, int kt) {
    constexpr int STG = decltype(stg)::value;
    const StagePtr cur{smem + STG * S::A_BYTES, smem + STG * S::B_BYTES};
    const StagePtr nxt{smem + (1 - STG) * S::A_BYTES, smem + (1 - STG) * S::B_BYTES};
    {
      auto dma = stage_dma(fast, kt + 1, 1 - STG);
      substep_with_loads<0, 1, GR, EARLY, D, S>(acc, af, bfr, cur, frags, dma, groups);
    }
#pragma unroll
    for (int kk = 1; kk < KK - 1; ++kk) {
      read_frags<S>(af[(kk + 1) & 1], bfr[(kk + 1) & 1], cur, frags, kk + 1);
      mfma_block<S::MB, S::NB>(acc, af[kk & 1], bfr[kk & 1]);
      sched_substep<S, A_KC, B_KC, true>();
    }
    // keep the barrier after every MFMA issued so far (the compiler would hoist it)
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<0>();
    __syncthreads();
    // stage kt is free now: it receives step kt + 2 (after the last step this reads
    // a stale stage; the values are never used)
    {
      auto dma = stage_dma(fast, kt + 2, STG);
      substep_with_loads<KK - 1, 0, GR, 0, EARLY, S>(acc, af, bfr, nxt, frags, dma, groups);
    }
  };
  int kt = 0;
  // iteration kt loads steps kt + 1 and kt + 2: both inside K while kt + 2 < nfull
  for (; kt + 3 < nfull; kt += 2) {
    step(Stage0(), Fast(), kt);
    step(Stage1(), Fast(), kt + 1);
  }
  // the rest, also in pairs: with an odd step count the last step computes on a
  // zero-filled stage and adds exact zeros
  for (; kt < nk; kt += 2) {
    step(Stage0(), Slow(), kt);
    step(Stage1(), Slow(), kt + 1);
  }
  // the zero fills issued under the last steps must land before the caller reuses LDS
  wait_vmcnt<0>();
  __syncthreads();
}

// ---------------------------------------------------------------------------
// An accumulator value read from its accumulation register where it is used (for
// values used once: left to itself, the register allocator moves the tile between
// register files and reads some values several times).
__device__ __forceinline__ float acc_read(float a) {
  float r;
  asm("v_accvgpr_read_b32 %0, %1" : "=v"(r) : "a"(a));
  return r;
}

}  // namespace flce
