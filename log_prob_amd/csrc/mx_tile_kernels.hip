// The head with 4-bit weights for many tokens (gfx950): logits, or log-prob partials, of
//
//   z[m, v] = scale * sum_k X[m, k] W[v, k],  X and W in MXFP4
//
// in 256 x 256 tiles through LDS, bound by the matrix pipe.  A code tile has the bytes of a
// bf16 tile of a quarter of the K, and an instruction the cycles of a bf16 one, so the
// direct-to-LDS pipeline is that of the bf16 kernels, with the scales as a third, small stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_mfma.h"

namespace flce {

namespace {

// Many tokens: 256 x 256 tiles, 4 waves of 128 x 128.
//
// The pipeline of the bf16 kernels, on code tiles: a step is 256 K, 128 bytes of codes a row
// (the bytes of 64 bf16), two stages of 64 KiB in LDS filled by direct-to-LDS loads, half of
// a step's loads issued right after the barrier that frees its stage and half under the next
// sub-step, and each sub-step's fragments read while the one before it computes.  Scales come
// 16 bytes of a row (two steps) at a time into two 8 KiB buffers of their own, and each lane
// reads a dword of them (its four blocks of a step) per 32-row fragment.
using MxShape = BigShape;                    // of the products and the epilogue
constexpr int MX_TILE_BYTES = 128 * 256;     // one operand's codes of a step
constexpr int MX_SCALE_BYTES = 16 * 256;     // one operand's scales of two steps
constexpr int MX_LDS = 4 * MX_TILE_BYTES + 4 * MX_SCALE_BYTES;
static_assert(MX_LDS <= 160 * 1024, "LDS");

// One operand tile: codes and scales of its first row, strides of the scales, rows that exist,
// columns.
struct MxTile {
  const uint8_t* codes;
  const uint8_t* scales;
  uint32_t row_stride, quad_stride;
  int valid;
  int H;
};

// Direct-to-LDS loads of a step's operand tile: 8 a wave, load j bringing rows 64 wave + 8 j
// .. + 7, lane i the 16 bytes of row i / 8 whose position is i % 8.  A lane's offset depends
// on j only through the swizzle (j % 4); the rows and the step move with the scalar offset.
// Both operands have the same rows of codes, so they share all of it.
struct MxCodeDma {
  uint32_t voff[4];
  uint32_t ld, row0;  // bytes of a row of codes; offset of the wave's first row
  int wave;
  __device__ __forceinline__ void init(int H, int wave_id) {
    wave = wave_id;
    ld = (uint32_t)mx_code_bytes(H, kMxFp4);
    row0 = 64u * (uint32_t)wave * ld;
    const uint32_t lane = threadIdx.x & 63, r = lane >> 3;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) voff[j] = r * ld + (((lane & 7) ^ r ^ j) << 4);
  }
  // load j of step st (byte offset 128 st) from the tile at rsrc to the LDS tile at lds.  FAST:
  // every row and chunk exists; otherwise rows past `valid` and chunks past `lim` are zeros.
  template <bool FAST>
  __device__ __forceinline__ void issue(const i32x4& rsrc, int valid, int lim, int st, int j,
                                        uint32_t lds) const {
    uint32_t v = voff[j & 3];
    if constexpr (!FAST) {
      const int lane = threadIdx.x & 63, r = lane >> 3;
      v = r + 64 * wave + 8 * j < valid && ((lane & 7) ^ r ^ (j & 3)) < lim ? v : OOB_OFFSET;
    }
    dma16<0>(rsrc, v, 128u * (uint32_t)st + row0 + 8u * (uint32_t)j * ld,
             lds + 8192u * (uint32_t)wave + 1024u * (uint32_t)j);
  }
};

// LDS byte offsets of a lane's fragments and scales, block 0 of the wave's rows from idx0.
struct MxFrag {
  uint32_t code[4];
  uint32_t scale;
  __device__ __forceinline__ void init(int idx0, int lane, uint32_t region, uint32_t scale_region) {
    const int r = idx0 + (lane & 31), half = lane >> 5;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
      code[kk] = region + (uint32_t)(r * 128 + (((4 * half + kk) ^ mx_swz(r)) << 4));
    scale = scale_region + (uint32_t)(16 * r + 4 * half);
  }
  __device__ __forceinline__ u32x4 read(const char* stage, int blk, int kk) const {
    return *reinterpret_cast<const u32x4*>(stage + code[kk] + 4096 * blk);
  }
  // parity: which of the pair's two steps
  __device__ __forceinline__ int read_scale(const char* pair, int blk, int parity) const {
    return *reinterpret_cast<const int*>(pair + scale + 512 * blk + 8 * parity);
  }
};

// Loads of an operand's scales: wave w brings rows 64 w .. + 63, a lane one row's 16 bytes: a
// contiguous kilobyte in the tiled form, a line each in the row-major one.
struct MxScaleDma {
  i32x4 rsrc;
  uint32_t voff, quad_stride, lds;
  int pairs;
  __device__ __forceinline__ void init(const MxTile& t, int wave, const char* lds0) {
    const int row = 64 * wave + (int)(threadIdx.x & 63);
    rsrc = make_rsrc_fixed(t.scales);
    voff = row < t.valid ? t.row_stride * (uint32_t)row : OOB_OFFSET;
    quad_stride = t.quad_stride;
    lds = lds_addr_of(lds0) + (uint32_t)(1024 * wave);
    pairs = (int)(mx_scale_bytes(t.H) / 16);
  }
  // steps 2 pair and 2 pair + 1 into buffer `pair % 2`; a pair past the end is all zeros
  __device__ __forceinline__ void issue(int pair) const {
    const bool live = pair < pairs;
    dma16<0>(rsrc, live ? voff : OOB_OFFSET, live ? quad_stride * (uint32_t)pair : 0u,
             lds + (uint32_t)((pair & 1) * 2 * MX_SCALE_BYTES));
  }
};

struct MxRegs {
  u32x4 a[2][4], b[2][4];  // fragments of sub-steps of either parity
  int sa[2][4], sb[2][4];  // scales of steps of either parity
};

// Group g of 16 of sub-step kk: one MFMA, every other group a fragment read
// of the next sub-step (RKK, of `stage`), and a share of the loads [JB, JE).
template <int kk, int RKK, int STG, int g, int JB, int JE, bool FAST, class Ops>
__device__ __forceinline__ void mx_group(f32x16 (&acc)[4][4], MxRegs& r, const char* stage,
                                         const MxFrag& fa, const MxFrag& fb, const Ops& dma) {
  constexpr int cur = kk & 1, nxt = cur ^ 1, mb = g / 4, nb = g % 4, D = JE - JB;
  if constexpr (g % 2 == 0) {
    constexpr int i = g / 2;
    if constexpr (i < 4) r.a[nxt][i] = fa.read(stage, i, RKK);
    else r.b[nxt][i - 4] = fb.read(stage, i - 4, RKK);
  }
  acc[mb][nb] = mx_mfma<kk>(r.a[cur][mb], r.b[cur][nb], acc[mb][nb], r.sa[STG][mb], r.sb[STG][nb]);
  if constexpr (g % 2 == 0) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  if constexpr (D > 0) {
    __builtin_amdgcn_sched_barrier(0);
    dma.template issue<FAST>(JB + g * D / 16, JB + (g + 1) * D / 16);
    __builtin_amdgcn_sched_barrier(0);
  }
}
template <int kk, int RKK, int STG, int JB, int JE, bool FAST, class Ops, int... G>
__device__ __forceinline__ void mx_substep(f32x16 (&acc)[4][4], MxRegs& r, const char* stage,
                                           const MxFrag& fa, const MxFrag& fb, const Ops& dma,
                                           std::integer_sequence<int, G...>) {
  (mx_group<kk, RKK, STG, G, JB, JE, FAST>(acc, r, stage, fa, fb, dma), ...);
}

// The loads of a step: 8 of B's tile (X, which more tiles share in L2), then 8 of A's.
struct MxLoads {
  const MxCodeDma& c;
  const i32x4 &ra, &rb;
  int va, vb, lim, st;
  uint32_t la, lb;
  template <bool FAST>
  __device__ __forceinline__ void issue(int j0, int j1) const {
#pragma unroll
    for (int j = j0; j < j1; ++j) {
      if (j < 8) c.issue<FAST>(rb, vb, lim, st, j, lb);
      else c.issue<FAST>(ra, va, lim, st, j - 8, la);
    }
  }
};

// acc[mb][nb] = the 32 x 32 block (32 mb, 32 nb) of the wave's 128 x 128 of A B^T.
__device__ __forceinline__ void mx_mainloop(f32x16 (&acc)[4][4], char* smem, const MxTile& A,
                                            const MxTile& B) {
  constexpr int D = 16, EARLY = D / 2;  // loads of a step
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int mb = 0; mb < 4; ++mb)
#pragma unroll
    for (int nb = 0; nb < 4; ++nb)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[mb][nb][e] = 0.f;
  const int blocks = (int)mx_blocks(A.H);  // chunks of a row
  const int nk = (blocks + 7) / 8;
  // steps that lie inside K, where every row of both tiles exists (else none)
  const int nfull = A.valid >= 256 && B.valid >= 256 ? blocks / 8 : 0;
  char* scale_lds = smem + 4 * MX_TILE_BYTES;  // buffers of a pair: A's rows, then B's
  MxCodeDma codes;
  codes.init(A.H, wave);
  const i32x4 ra = make_rsrc_fixed(A.codes), rb = make_rsrc_fixed(B.codes);
  MxScaleDma da, db;
  da.init(A, wave, scale_lds);
  db.init(B, wave, scale_lds + MX_SCALE_BYTES);
  MxFrag fa, fb;
  fa.init((wave / 2) * 128, lane, 0u, 0u);
  fb.init((wave % 2) * 128, lane, 2u * MX_TILE_BYTES, (uint32_t)MX_SCALE_BYTES);
  // loads of step st into stage s (A0, A1, B0, B1); a step past K only zero-fills it
  const uint32_t lds0 = lds_addr_of(smem);
  auto loads = [&](int st, int s) {
    const int lim = min(max(blocks - 8 * st, 0), 8);
    return MxLoads{codes, ra, rb, A.valid, B.valid, lim, lim > 0 ? st : 0,
                   lds0 + (uint32_t)(s * MX_TILE_BYTES), lds0 + (uint32_t)((2 + s) * MX_TILE_BYTES)};
  };
  using Slow = std::integral_constant<bool, false>;
  using Fast = std::integral_constant<bool, true>;
  using Stage0 = std::integral_constant<int, 0>;
  using Stage1 = std::integral_constant<int, 1>;
  MxRegs r;
  auto read_scales = [&](int st, int set) {
    const char* pair = scale_lds + ((st >> 1) & 1) * 2 * MX_SCALE_BYTES;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.sa[set][i] = fa.read_scale(pair, i, set);
      r.sb[set][i] = fb.read_scale(pair, i, set);
    }
  };
  // prologue: the first pair's scales, step 0, and the early loads of step 1
  da.issue(0);
  db.issue(0);
  loads(0, 0).issue<false>(0, D);
  loads(1, 1).issue<false>(0, EARLY);
  wait_vmcnt<EARLY>();
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.a[0][i] = fa.read(smem, i, 0);
    r.b[0][i] = fb.read(smem, i, 0);
  }
  read_scales(0, 0);
  constexpr auto groups = std::make_integer_sequence<int, 16>();
  // step kt from stage STG (kt % 2 == STG)
  auto step = [&](auto stg, auto fast, int kt) {
    constexpr int STG = decltype(stg)::value;
    constexpr bool FAST = decltype(fast)::value;
    const char* cur = smem + STG * MX_TILE_BYTES;
    const char* nxt = smem + (1 - STG) * MX_TILE_BYTES;
    {
      const auto dma = loads(kt + 1, 1 - STG);
      mx_substep<0, 1, STG, EARLY, D, FAST>(acc, r, cur, fa, fb, dma, groups);
      mx_substep<1, 2, STG, 0, 0, FAST>(acc, r, cur, fa, fb, dma, groups);
      mx_substep<2, 3, STG, 0, 0, FAST>(acc, r, cur, fa, fb, dma, groups);
    }
    // keep the barrier after every MFMA issued so far (the compiler would hoist it)
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<0>();
    __syncthreads();
    // the stage of step kt is free: it receives step kt + 2, and after an even step the pair
    // buffer that held steps kt - 2 and kt - 1 receives the scales of kt + 2 and kt + 3
    {
      if constexpr (STG == 0) {
        da.issue((kt >> 1) + 1);
        db.issue((kt >> 1) + 1);
      }
      read_scales(kt + 1, 1 - STG);
      __builtin_amdgcn_sched_barrier(0);
      const auto dma = loads(kt + 2, STG);
      mx_substep<3, 0, STG, 0, EARLY, FAST>(acc, r, nxt, fa, fb, dma, groups);
    }
  };
  int kt = 0;
  for (; kt + 3 < nfull; kt += 2) {
    step(Stage0(), Fast(), kt);
    step(Stage1(), Fast(), kt + 1);
  }
  for (; kt + 1 < nk; kt += 2) {
    step(Stage0(), Slow(), kt);
    step(Stage1(), Slow(), kt + 1);
  }
  if (kt < nk) step(Stage0(), Slow(), kt);
  // the zero fills issued under the last steps must land before the caller reuses LDS
  wait_vmcnt<0>();
  __syncthreads();
}

// The tile of vocabulary rows (A) and tokens (B) of a workgroup.
__device__ __forceinline__ void mx_tile_product(f32x16 (&acc)[4][4], char* smem, const MxOperand& x,
                                                const MxOperand& w, int M, int H, int V, int mt, int vt) {
  const long code_ld = mx_code_bytes(H, kMxFp4);
  const int row0 = mt * 256, col0 = vt * 256;
  const MxTile A{w.codes + col0 * code_ld, w.scales + vt * w.layout.tile_stride,
                 (uint32_t)w.layout.row_stride, (uint32_t)w.layout.quad_stride, V - col0, H};
  const MxTile B{x.codes + row0 * code_ld, x.scales + mt * x.layout.tile_stride,
                 (uint32_t)x.layout.row_stride, (uint32_t)x.layout.quad_stride, M - row0, H};
  mx_mainloop(acc, smem, A, B);
}

// f: the sizes, outputs and queues that the tile loop and the epilogue of the bf16 forward use.
struct MxTileFwdArgs {
  MxOperand x, w;
  FwdTileArgs f;
};
template <bool ENT>
__global__ __launch_bounds__(256, 1) void mx_tile_fwd_kernel(MxTileFwdArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[MX_LDS];
  const int L = tile_claim(a.f.n_mt * a.f.n_vt, a.f.tq);
  if (L < 0) return;
  int mt, vt;
  group_coords(L, a.f.n_mt, a.f.n_vt, FWD_GROUP_M, mt, vt);
  f32x16 acc[4][4];
  mx_tile_product(acc, smem, a.x, a.w, a.f.M, a.f.H, a.f.V, mt, vt);
  fwd_epilogue<MxShape, ENT>(acc, smem, a.f, mt, vt);
}

// Logits of a tile: a lane holds 4 consecutive vocabulary entries of a token at a time.  Each
// wave turns its 128 x 128 block around in a 16 KiB slice of its own, 32 tokens at a time (no
// workgroup barrier): rows of 128 entries, 16-byte chunks swizzled by token, then whole rows
// to memory, 16 bytes a lane.  VEC: every row starts and ends at a multiple of 16 bytes, and the
// stores carry the non-temporal hint (4096 x 32768 bf16 logits over H = 4096: 297 -> 281 us).
// Otherwise they are unaligned ones without it, for a neighbouring tile's store may fill the
// rest of a line, and a row's last entries go one by one (1000 x 50257 over H = 2048: 92 us in
// bf16 and 103 in fp32; element by element throughout, 136 and 134).
template <class T, bool VEC>
__global__ __launch_bounds__(256, 1) void mx_tile_logits_kernel(MxLogitsArgs p) {
  __shared__ __attribute__((aligned(1024))) char smem[MX_LDS];
  int mt, vt;
  tile_coords((int)blockIdx.x, p.n_mt * p.n_vt, p.n_mt, p.n_vt, FWD_GROUP_M, mt, vt);
  f32x16 acc[4][4];
  mx_tile_product(acc, smem, p.x, p.w, p.M, p.H, p.V, mt, vt);
  constexpr int ES = (int)sizeof(typename T::mem), RB = 128 * ES, CH = RB / 16;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lc = lane & 31, half = lane >> 5;
  const int v0 = vt * 256 + (wave / 2) * 128, t0 = mt * 256 + (wave % 2) * 128;
  char* slice = smem + wave * 16384;
  typename T::mem* out = static_cast<typename T::mem*>(p.out);
#pragma unroll
  for (int nb = 0; nb < 4; ++nb) {
#pragma unroll
    for (int mb = 0; mb < 4; ++mb)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // entries 32 mb + 8 q + 4 half .. + 3 of token lc
        float d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = p.scale * acc[mb][nb][4 * q + i];
        if constexpr (ES == 4) {
          const int c = 8 * mb + 2 * q + half;
          *reinterpret_cast<f32x4_t*>(slice + lc * RB + ((c ^ lc) << 4)) = f32x4_t{d[0], d[1], d[2], d[3]};
        } else {
          const int c = 4 * mb + q;
          *reinterpret_cast<u32x2*>(slice + lc * RB + ((c ^ (lc & 15)) << 4) + 8 * half) =
              u32x2{pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3])};
        }
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    constexpr int RPI = 64 / CH, E = 16 / ES;  // rows an instruction, entries a lane
#pragma unroll
    for (int it = 0; it < 32 / RPI; ++it) {
      const int r = it * RPI + lane / CH, c = lane % CH;
      const u32x4 v = *reinterpret_cast<const u32x4*>(slice + r * RB + ((c ^ (r & (CH - 1))) << 4));
      const int t = t0 + 32 * nb + r, col = v0 + c * E;
      typename T::mem* to = out + (long)t * p.ldo + col;
      if (t >= p.M || col >= p.V) continue;
      if constexpr (VEC) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(to));
      else store_entries<T>(to, v, p.V - col);
    }
    // the slice's reads have returned before the next 32 tokens overwrite it
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// VEC: rows and columns in multiples of 16 bytes.
template <class T>
void tile_logits(const MxLogitsArgs& a, hipStream_t s) {
  constexpr int E = 16 / (int)sizeof(typename T::mem);
  const bool vec = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.ldo % E == 0 && a.V % E == 0;
  const unsigned g = (unsigned)((int64_t)a.n_mt * a.n_vt);
  if (vec) mx_tile_logits_kernel<T, true><<<g, 256, 0, s>>>(a);
  else mx_tile_logits_kernel<T, false><<<g, 256, 0, s>>>(a);
}

}  // namespace

hipError_t launch_mx_tile_logits(const MxLogitsArgs& a, hipStream_t s) {
  if (a.out_dtype == kBf16) tile_logits<Bf16>(a, s);
  else tile_logits<F32>(a, s);
  return hipGetLastError();
}

hipError_t launch_mx_tile_fwd(const MxFwdArgs& a, TileQueue tq, hipStream_t s) {
  const int64_t n = (int64_t)a.n_mt * a.n_vt;
  const QueueShape qs = queue_shape(n);
  MxTileFwdArgs b{};
  b.x = a.x;
  b.w = a.w;
  b.f.M = a.M;
  b.f.H = a.H;
  b.f.V = a.V;
  b.f.scale = a.scale;
  b.f.n_mt = a.n_mt;
  b.f.n_vt = a.n_vt;
  b.f.Mpad = (int)a.tile_stride;
  b.f.part_m = a.part_m;
  b.f.part_s = a.part_s;
  b.f.part_u = a.part_u;
  b.f.tq = tq;
  b.f.tq.queue = qs.queue;
  const unsigned g = (unsigned)(n + qs.spare);
  if (a.part_u) mx_tile_fwd_kernel<true><<<g, 256, 0, s>>>(b);
  else mx_tile_fwd_kernel<false><<<g, 256, 0, s>>>(b);
  return hipGetLastError();
}

}  // namespace flce
