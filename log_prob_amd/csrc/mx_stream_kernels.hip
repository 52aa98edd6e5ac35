// The head with 4-bit weights for few tokens (gfx950), and the merge of log-prob partials.
//
//   z[m, v] = scale * sum_k X[m, k] W[v, k],  X and W in MXFP4
//
// With up to 128 tokens the kernel is bound by memory: W's codes and scales are read once.
// They come through a ring of LDS stages by direct-to-LDS loads, 128 contiguous bytes of a row
// for 8 lanes, ahead of the products (loaded straight into the matrix instruction's registers,
// 16 bytes a lane from 32 rows at once, one token over 151936 x 2048 took 60 us).  Two
// workgroups of four waves share a compute unit where each takes 128 vocabulary rows, so a stage
// has 32 KiB at most (one workgroup and three stages for 128 tokens: 65 us over 151936 x 2048
// instead of 48); with fewer rows and more than 8 tokens the stages fill half of the LDS and
// more, and one runs (StreamCfg<2, 2, 32>, <1, 4, 32> and <2, 2, 64>: 84, 104 and 100 KiB).
// More tokens run in tiles of up to 128.  A round of 510 such tiles (288 x 21760, 128 x 96, two
// a unit) takes 6.3 us and 0.9 to 1.05 us for each 256 K, in which a unit loads 57 KB to LDS, 24
// bytes a clock, and its matrix pipe works for a third of the cycles: neither is at its limit.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_mfma.h"

namespace flce {

namespace {

// A workgroup of RW x KW = 4 waves takes 32 RW vocabulary rows; wave (rw, kw) multiplies rows
// 32 rw .. + 31 over every KW-th 256 K, and the KW partial products meet in LDS at the end
// (fewer rows a workgroup where the vocabulary is too small to fill the chip otherwise).  XR
// token rows are staged (8, or 32 TB); or none (XR = 0): the few tokens of a decoding step are
// quantised by every workgroup for itself while its first rows of W are on their way, which
// spares the launch that would do it (at most kMxOwnBytes of codes).
template <int RW_, int KW_, int XR_>
struct StreamCfg {
  static constexpr int RW = RW_, KW = KW_, XR = XR_;
  static constexpr bool OWN = XR == 0;
  static constexpr int TB = XR <= 32 ? 1 : XR / 32;       // 32-token blocks
  static constexpr int ROWS = 32 * RW;                    // vocabulary rows
  static constexpr int W_BYTES = KW * ROWS * 128, X_BYTES = KW * XR * 128;
  static constexpr int STAGE = W_BYTES + X_BYTES;
  static constexpr int NS = XR > 64 ? 2 : 3;              // stages
  static constexpr int W_LOADS = W_BYTES / 4096;                       // a wave, 1 KiB each
  static constexpr int X_LOADS = (X_BYTES + 4095) / 4096;
  static constexpr int LOADS = W_LOADS + X_LOADS;
  // scales: SP 16-byte pieces of a row (of two steps each) at a time, double-buffered
  static constexpr int SP = XR >= 64 ? 1 : 4, SCALE_STEPS = 2 * SP, SCALE_LD = 16 * SP;
  static constexpr int LOAD_ROWS = 64 / SP;                            // rows of a load
  static constexpr int SCALE_ROWS = ROWS + (OWN ? 0 : XR < 16 ? 16 : XR);
  static constexpr int SCALE_BUF = (SCALE_ROWS + LOAD_ROWS - 1) / LOAD_ROWS * 1024;
  static constexpr int SCALE_LOADS = (SCALE_BUF / 1024 + 3) / 4;       // a wave, at most
  static constexpr int OWN_AT = NS * STAGE + 2 * SCALE_BUF;            // own codes, then scales
  static constexpr int LDS = OWN_AT + (OWN ? kMxOwnBytes + kMxOwnBytes / 8 : 0);
  static constexpr int MB = 1, NB = TB;  // as lane_col_max and lane_col_sums name them
  static_assert(RW * KW == 4 && W_BYTES == 16384, "four waves");
  static_assert(LDS <= (KW == 1 ? 80 : 160) * 1024, "LDS; two a compute unit with 128 rows each");
};

// Order of a step's products: one product a time, each but the last block's with a read of the
// next block's (and its scales first).
template <int... I>
__device__ __forceinline__ void among(std::integer_sequence<int, I...>) {
  constexpr int N = (int)sizeof...(I);
  ((I < N - 4 ? __builtin_amdgcn_sched_group_barrier(0x100, I % 4 == 0 ? 2 : 1, 0) : (void)0,
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0)),
   ...);
}

// acc[0][tb]: the wave's 32 vocabulary rows x token block tb, as (A = W, B = X) for the
// log-probs (a lane then holds 16 vocabulary rows of one token) and as (A = X, B = W) for the
// logits (a lane holds one vocabulary column, so a store covers 128 contiguous bytes of a
// row).  Summed over the KW waves of the same rows, in order, in the waves with kw = 0.
template <class C, bool LOGITS>
__device__ __forceinline__ void stream_product(f32x16 (&acc)[1][C::TB], char* smem, const uint16_t* X,
                                               const MxOperand& x, const MxOperand& w, int M, int H,
                                               int V, int v0, int m0) {
  constexpr int RW = C::RW, KW = C::KW, TB = C::TB, NS = C::NS;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rw = wave % RW, kw = wave / RW;
  const uint32_t ld = (uint32_t)mx_code_bytes(H, kMxFp4);
  const int blocks = (int)mx_blocks(H), steps = (blocks + 7) / 8, nk = (steps + KW - 1) / KW;
  const uint32_t lds0 = lds_addr_of(smem);
  const i32x4 wr = make_rsrc_fixed(w.codes + (long)v0 * ld), xr = make_rsrc_fixed(x.codes + (long)m0 * ld);
  const int wvalid = V - v0;
  M -= m0;

  // loads of stage k (steps KW k .. + KW - 1): load i covers rows 8 (i % n) .. + 7 of step
  // KW k + i / n; lane l row l / 8, the chunk whose position is l % 8
  const int lr = lane >> 3, lp = lane & 7;
  auto issue = [&](int k, int slot) {
    const uint32_t st = lds0 + (uint32_t)(slot * C::STAGE);
#pragma unroll
    for (int q = 0; q < C::W_LOADS; ++q) {
      const int i = wave * C::W_LOADS + q, sub = i / (C::ROWS / 8), r = 8 * (i % (C::ROWS / 8)) + lr;
      const int b = 8 * (KW * k + sub) + (lp ^ mx_swz(r));
      const bool ok = r < wvalid && b < blocks;
      dma16<0>(wr, ok ? (uint32_t)r * ld + 16u * (uint32_t)b : OOB_OFFSET, 0u, st + 1024u * (uint32_t)i);
    }
    if constexpr (!C::OWN) {
#pragma unroll
      for (int q = 0; q < C::X_LOADS; ++q) {
        const int i = wave * C::X_LOADS + q, sub = i / (C::XR / 8), r = 8 * (i % (C::XR / 8)) + lr;
        const int b = 8 * (KW * k + sub) + (lp ^ mx_swz(r));
        const bool ok = r < M && b < blocks;
        // (fewer loads than waves: the waves without one repeat it with nothing to bring)
        if (C::X_BYTES >= 4096 || i < C::X_BYTES / 1024)
          dma16<0>(xr, ok ? (uint32_t)r * ld + 16u * (uint32_t)b : OOB_OFFSET, 0u,
                   st + (uint32_t)C::W_BYTES + 1024u * (uint32_t)i);
        else
          dma16<0>(xr, OOB_OFFSET, 0u, lds0 + (uint32_t)(C::NS * C::STAGE + 2 * C::SCALE_BUF));
      }
    }
  };
  // scales of SCALE_STEPS steps, chunk c: lane l row l / SP, 16-byte piece l % SP
  const int pieces = (int)(mx_scale_bytes(H) / 16);
  const i32x4 ws = make_rsrc_fixed(w.scales + mx_scale_row(w.layout, v0)), xs = make_rsrc_fixed(x.scales + mx_scale_row(x.layout, m0));
  const uint32_t sld = (uint32_t)mx_scale_bytes(H);
  auto issue_scales = [&](int c) {
    const uint32_t buf = lds0 + (uint32_t)(NS * C::STAGE + (c & 1) * C::SCALE_BUF);
#pragma unroll
    for (int q = 0; q < C::SCALE_LOADS; ++q) {
      const int i = 4 * q + wave;  // wave-uniform
      if (i < C::SCALE_BUF / 1024) {
        const int r = C::LOAD_ROWS * i + lane / C::SP, p = C::SP * c + lane % C::SP;
        // (a load's rows are all of W or all of X)
        const bool is_w = C::LOAD_ROWS * i < C::ROWS;
        const int rr = is_w ? r : r - C::ROWS;
        const bool ok = rr < (is_w ? wvalid : M) && p < pieces;
        dma16<0>(C::OWN || is_w ? ws : xs, ok ? (uint32_t)rr * sld + 16u * (uint32_t)p : OOB_OFFSET, 0u,
                 buf + 1024u * (uint32_t)i);
      }
    }
  };

  // fragments: the wave's row of W and of each token block (rows past XR repeat earlier ones)
  const int half = lane >> 5, r = lane & 31;
  uint32_t wf[4], xf[4];
  const int xrow = C::OWN ? (r < M ? r : 0) : r & (C::XR - 1);
  const int own_ld = 128 * KW * nk;  // bytes of a row of own codes: every step, and an 8th of scales
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    wf[kk] = (uint32_t)(kw * C::ROWS * 128 + (32 * rw + r) * 128 + (((4 * half + kk) ^ mx_swz(r)) << 4));
    xf[kk] = C::OWN ? (uint32_t)(C::OWN_AT + xrow * own_ld + 128 * kw + ((4 * half + kk) << 4))
                    : (uint32_t)(C::W_BYTES + kw * C::XR * 128 + xrow * 128 +
                                 (((4 * half + kk) ^ mx_swz(xrow)) << 4));
  }
  const uint32_t wsf = (uint32_t)((32 * rw + r) * C::SCALE_LD + 4 * half);
  const uint32_t xsf = C::OWN ? (uint32_t)(C::OWN_AT + kMxOwnBytes + xrow * (own_ld / 16) + 8 * kw + 4 * half)
                              : (uint32_t)((C::ROWS + xrow) * C::SCALE_LD + 4 * half);
#pragma unroll
  for (int tb = 0; tb < TB; ++tb)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[0][tb][e] = 0.f;

  issue_scales(0);
#pragma unroll
  for (int k = 0; k < NS - 1; ++k) issue(k, k);
  if constexpr (C::OWN) {
    // thread t takes chunks of 8 elements t, t + 256, ...; whole steps, zeros past H (the first
    // barrier of the loop publishes them)
    const int chunks = own_ld / 4;
    for (int i = threadIdx.x; i < M * chunks; i += 256) {
      const int m = i / chunks, c = i - m * chunks;
      float v[8];
      load8<Bf16, true>(X + (long)m * H, 8 * c, H, v);
      const uint32_t byte = mx_scale_byte<kMxFp4>(v);
      *reinterpret_cast<uint32_t*>(smem + C::OWN_AT + 4 * i) = mx_encode<kMxFp4>(v, byte).x;
      if ((c & 3) == 0) smem[C::OWN_AT + kMxOwnBytes + i / 4] = (char)byte;
    }
  }
  int slot = 0;
  for (int k = 0; k < nk; ++k) {
    // stage k has landed (the loads of the NS - 2 stages after it may be in flight), and
    // every wave is done with stage k - 1, whose slot the next loads take
    wait_vmcnt<C::LOADS*(NS - 2)>();
    __syncthreads();
    const int c = KW * k / C::SCALE_STEPS;
    if (KW * k % C::SCALE_STEPS == 0) issue_scales(c + 1);
    issue(k + NS - 1, slot == 0 ? NS - 1 : slot - 1);
    const char* st = smem + slot * C::STAGE;
    const char* sb = smem + NS * C::STAGE + (c & 1) * C::SCALE_BUF + 8 * ((KW * k + kw) & (C::SCALE_STEPS - 1));
    const int sw = *reinterpret_cast<const int*>(sb + wsf);
    u32x4 wv[4], xv[2][4];
    int sx[2];
    auto read_x = [&](int tb) {
      sx[tb & 1] =
          *reinterpret_cast<const int*>(C::OWN ? smem + xsf + 8 * KW * k : sb + xsf + 32 * C::SCALE_LD * tb);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        xv[tb & 1][kk] = *reinterpret_cast<const u32x4*>(C::OWN ? smem + xf[kk] + 128 * KW * k
                                                                : st + xf[kk] + 4096 * tb);
    };
    auto product = [&](auto kk, int tb) {
      constexpr int K = decltype(kk)::value;
      const int b = tb & 1;
      acc[0][tb] = LOGITS ? mx_mfma<K>(xv[b][K], wv[K], acc[0][tb], sx[b], sw)
                          : mx_mfma<K>(wv[K], xv[b][K], acc[0][tb], sw, sx[b]);
    };
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) wv[kk] = *reinterpret_cast<const u32x4*>(st + wf[kk]);
    read_x(0);
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
      if (tb + 1 < TB) read_x(tb + 1);
      product(std::integral_constant<int, 0>(), tb);
      product(std::integral_constant<int, 1>(), tb);
      product(std::integral_constant<int, 2>(), tb);
      product(std::integral_constant<int, 3>(), tb);
    }
    // the first block's ten reads, then each block's products among the reads of the next
    __builtin_amdgcn_sched_group_barrier(0x100, 10, 0);
    among(std::make_integer_sequence<int, 4 * TB>());
    slot = slot == NS - 1 ? 0 : slot + 1;
  }
  // the zero fills of the stages past the end must land before the LDS is used again
  wait_vmcnt<0>();
  __syncthreads();
  if constexpr (KW > 1) {
    float* join = reinterpret_cast<float*>(smem);  // [kw - 1][rw][tb][e][lane]
    if (kw > 0) {
#pragma unroll
      for (int tb = 0; tb < TB; ++tb)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          join[(((kw - 1) * RW + rw) * TB + tb) * 1024 + 64 * e + lane] = acc[0][tb][e];
    }
    __syncthreads();
    if (kw == 0) {
#pragma unroll
      for (int j = 0; j < KW - 1; ++j)
#pragma unroll
        for (int tb = 0; tb < TB; ++tb)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[0][tb][e] += join[((j * RW + rw) * TB + tb) * 1024 + 64 * e + lane];
    }
  }
}

// The vocabulary rows and tokens of a workgroup.
template <class C>
__device__ __forceinline__ void stream_coords(int M, int V, int& mt, int& vt) {
  mt = 0;
  vt = (int)blockIdx.x;
  if constexpr (C::XR >= 64) {
    const int n_mt = (M + 32 * C::TB - 1) / (32 * C::TB), n_vt = (V + C::ROWS - 1) / C::ROWS;
    tile_coords((int)blockIdx.x, n_mt * n_vt, n_mt, n_vt, FWD_GROUP_M, mt, vt);
  }
}

// The staging LDS, and a kilobyte that loads with nothing to bring may zero.
template <class C>
constexpr int stream_lds = C::LDS + (!C::OWN && C::X_BYTES < 4096 ? 1024 : 0);

template <class C, class T>
__global__ __launch_bounds__(256) void mx_stream_logits_kernel(MxLogitsArgs p) {
  __shared__ __attribute__((aligned(1024))) char smem[stream_lds<C>];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int mt, vt;
  stream_coords<C>(p.M, p.V, mt, vt);
  const int v0 = vt * C::ROWS, m0 = mt * 32 * C::TB;
  f32x16 acc[1][C::TB];
  stream_product<C, true>(acc, smem, p.X, p.x, p.w, p.M, p.H, p.V, v0, m0);
  typename T::mem* out = static_cast<typename T::mem*>(p.out);
  if constexpr (C::XR < 64) {
    const int v = v0 + 32 * (wave % C::RW) + (lane & 31);
    if (wave / C::RW != 0 || v >= p.V) return;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int m = m0 + acc_row(lane, e);
      if (m < p.M) out[(long)m * p.ldo + v] = T::from_f32(p.scale * acc[0][0][e]);
    }
  } else {
    // many tokens: through LDS to rows of ROWS entries, 16 bytes a lane
    constexpr int ES = (int)sizeof(typename T::mem), LD = C::ROWS * ES + 16, E = 16 / ES, CH = C::ROWS / E;
    constexpr int JOIN = (C::KW - 1) * C::RW * C::TB * 4096;  // what the KW waves exchanged
    static_assert(JOIN + 32 * C::TB * LD <= C::LDS, "staging");
    char* tile = smem + JOIN;
    if (wave / C::RW == 0) {
#pragma unroll
      for (int tb = 0; tb < C::TB; ++tb)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          *reinterpret_cast<typename T::mem*>(tile + (32 * tb + acc_row(lane, e)) * LD +
                                              (32 * (wave % C::RW) + (lane & 31)) * ES) =
              T::from_f32(p.scale * acc[0][tb][e]);
    }
    __syncthreads();
    const int rows = p.M - m0 < 32 * C::TB ? p.M - m0 : 32 * C::TB;
    for (int i = threadIdx.x; i < rows * CH; i += 256) {
      const int r = i / CH, c = i % CH, v = v0 + c * E;
      const u32x4 d = *reinterpret_cast<const u32x4*>(tile + r * LD + 16 * c);
      if (v < p.V) store_entries<T>(out + (long)(m0 + r) * p.ldo + v, d, p.V - v);
    }
  }
}

// Partials of the workgroup's vocabulary rows: maximum, then the shifted sums, each over the
// lane's 16 rows, the two half-waves and the RW waves.
template <class C, bool ENT>
__global__ __launch_bounds__(256) void mx_stream_fwd_kernel(MxFwdArgs p) {
  constexpr int RW = C::RW, TB = C::TB, TT = 32 * TB;
  __shared__ __attribute__((aligned(1024))) char smem[stream_lds<C>];
  static_assert((3 * RW + (C::KW - 1) * RW * 32) * TT * 4 <= C::LDS, "epilogue buffers");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rw = wave % RW, kw = wave / RW, lc = lane & 31;
  int mt, vt;
  stream_coords<C>(p.M, p.V, mt, vt);
  const int v0 = vt * C::ROWS, m0 = mt * TT;
  f32x16 acc[1][TB];
  stream_product<C, false>(acc, smem, p.X, p.x, p.w, p.M, p.H, p.V, v0, m0);
  // [rw][token] maxima and sums, behind what the KW waves exchanged
  float* red = reinterpret_cast<float*>(smem) + (C::KW - 1) * RW * TB * 1024;
  float* comb = red + RW * TT;
  const float c1 = p.scale * LOG2E, ac1 = fabsf(c1);
  const int vrows = p.V - v0 - 32 * rw;  // of the wave; those past it are masked
  if (kw == 0) {
    float mx[TB];
    if (c1 >= 0.f) lane_col_max<false, true, C>(acc, lane, vrows, mx);
    else lane_col_max<true, true, C>(acc, lane, vrows, mx);
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
      const float m = halves_reduce(mx[tb], mx[tb], [](float x, float y) { return max_raw(x, y); });
      if (lane < 32) red[rw * TT + 32 * tb + lc] = m;
    }
  }
  __syncthreads();
  if (kw == 0) {
    float nm2[TB], sv[TB], uv[TB];
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
      float m = red[32 * tb + lc];
#pragma unroll
      for (int k = 1; k < RW; ++k) m = fmaxf(m, red[k * TT + 32 * tb + lc]);
      nm2[tb] = -ac1 * m;
    }
    lane_col_sums<ENT, true, C>(acc, lane, vrows, c1, nm2, sv, uv);
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
      const float s = halves_reduce(sv[tb], sv[tb], [](float x, float y) { return x + y; });
      const float u = halves_reduce(uv[tb], uv[tb], [](float x, float y) { return x + y; });
      if (lane < 32) {
        comb[rw * TT + 32 * tb + lc] = s;
        comb[(RW + rw) * TT + 32 * tb + lc] = u;
      }
    }
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t < TT && m0 + t < p.M) {
    float m = red[t], s = comb[t], u = comb[RW * TT + t];
#pragma unroll
    for (int k = 1; k < RW; ++k) {
      m = fmaxf(m, red[k * TT + t]);
      s += comb[k * TT + t];
      u += comb[(RW + k) * TT + t];
    }
    const long off = (long)vt * p.tile_stride + (m0 + t) * p.token_stride;
    p.part_m[off] = ac1 * m * LN2;
    p.part_s[off] = s;
    if constexpr (ENT) p.part_u[off] = u * LN2;
  }
}

// The configuration for M tokens of a call that takes `rows` vocabulary rows a workgroup
// (mx_stream_rows); own: X has not been quantised.  Tiles of 64 tokens, three stages deep, where
// all are resident at once or the workgroup takes 64 vocabulary rows; else of 96 or 128, of two
// stages, which load less for each product
// (300 x 4096 x 4000 logits: 15 against 19 us; 600 x 1600 x 50257: 72 against 59 us).
template <int XR, class F>
void with_cfg(int rows, F f) {
  if (rows == 128) f(StreamCfg<4, 1, XR>());
  if constexpr (XR <= 64) {
    if (rows == 64) f(StreamCfg<2, 2, XR>());
  }
  if constexpr (XR <= 32) {
    if (rows == 32) f(StreamCfg<1, 4, XR>());
  }
}
template <class F>
void with_tokens(int M, int V, bool own, int rows, F f) {
  if (own) with_cfg<0>(rows, f);
  else if (M <= 8) with_cfg<8>(rows, f);
  else if (M <= 32) with_cfg<32>(rows, f);
  else if (M <= 64 || rows == 64 || (V + 127) / 128 * (int64_t)((M + 63) / 64) <= kMxStreamResident)
    with_cfg<64>(rows, f);
  else if ((M + 127) / 128 * 96 >= M) with_cfg<96>(rows, f);
  else with_cfg<128>(rows, f);
}

// ---------------------------------------------------------------------------
// Merge: per token, the target logit as a dot product of codes, then m* = max m_j,
// S = sum s_j e^(m_j - m*), U = sum e^(m_j - m*) (u_j + (m_j - m*) s_j) over the vocabulary
// tiles j; lse = m* + log S, logprob = min(z_t - lse, 0), entropy = max(log S - U / S, 0) (the
// bounds hold exactly: fp32 rounding can put a value next to one a few ulps past it; a NaN in
// the row's sums or its target logit passes them).
// ROWS tokens a workgroup: 16 where the tokens of a vocabulary tile are contiguous (64-byte
// pieces, and a token's tiles over 32 threads), or 4 where that would leave most of the chip
// idle; one where a token's tiles are contiguous.
constexpr int MERGE_THREADS = 512;
template <int ROWS, bool ENT>
__global__ __launch_bounds__(MERGE_THREADS) void mx_merge_kernel(MxFwdArgs p) {
  constexpr int SLICES = MERGE_THREADS / ROWS, WAVES = MERGE_THREADS / 64;
  __shared__ float sm[2][SLICES][ROWS];
  __shared__ float zt[ROWS < WAVES ? WAVES : ROWS];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const long row0 = (long)blockIdx.x * ROWS;
  const long code_ld = mx_code_bytes(p.H, kMxFp4);
  auto scale = [](const MxOperand& o, long r, int b) -> uint32_t {
    return o.scales[mx_scale_row(o.layout, r) + (b >> 4) * o.layout.quad_stride + (b & 15)];
  };
  // target logits: a wave a token (one token: its blocks over all waves); a block's sum of
  // code products is exact, its two scales multiply it as one (with X's largest blocks against
  // W's smallest, one after the other passed fp32's range on the way)
  for (int i = ROWS == 1 ? 0 : wave; i < ROWS; i += WAVES) {
    const long row = row0 + i;
    const int64_t t = row < p.M ? p.targets[row] : -1;
    float s = 0.f;
    const bool valid = row < p.M && t != p.ignore_index && t >= 0 && t < p.V;
    if (ROWS == 1 && valid && p.X) {
      // X not quantised beforehand: a chunk of 8 elements a thread
      for (int c = threadIdx.x; c < 4 * (int)mx_blocks(p.H); c += MERGE_THREADS) {
        float v[8], xv[8], wv[8];
        load8<Bf16, true>(p.X + row * p.H, 8 * c, p.H, v);
        const uint32_t byte = mx_scale_byte<kMxFp4>(v);
        mx_decode<kMxFp4>(mx_encode<kMxFp4>(v, byte), 127u, xv);
        mx_decode<kMxFp4>(u32x2_t{*reinterpret_cast<const uint32_t*>(p.w.codes + t * code_ld + 4l * c), 0u},
                          127u, wv);
        float d = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) d = fmaf(xv[j], wv[j], d);
        s += mx_scale_product(d, byte, scale(p.w, t, c >> 2));
      }
    } else if (valid) {
      for (int b = ROWS == 1 ? (int)threadIdx.x : lane; b < (int)mx_blocks(p.H);
           b += ROWS == 1 ? MERGE_THREADS : 64) {
        const u32x4 xc = *reinterpret_cast<const u32x4*>(p.x.codes + row * code_ld + 16l * b);
        const u32x4 wc = *reinterpret_cast<const u32x4*>(p.w.codes + t * code_ld + 16l * b);
        float d = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float xv[8], wv[8];
          mx_decode<kMxFp4>(u32x2_t{xc[k], 0u}, 127u, xv);
          mx_decode<kMxFp4>(u32x2_t{wc[k], 0u}, 127u, wv);
#pragma unroll
          for (int j = 0; j < 8; ++j) d = fmaf(xv[j], wv[j], d);
        }
        s += mx_scale_product(d, scale(p.x, row, b), scale(p.w, t, b));
      }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
    if (lane == 0) zt[ROWS == 1 ? wave : i] = s * p.scale;
  }
  const int lr = threadIdx.x % ROWS, sl = threadIdx.x / ROWS;
  const long row = row0 + lr;
  const bool live = row < p.M;
  const float* pm = p.part_m + row * p.token_stride;
  const float* ps = p.part_s + row * p.token_stride;
  float m = -INFINITY;
  if (live) {
#pragma unroll 4
    for (int j = sl; j < p.n_vt; j += SLICES) m = fmaxf(m, pm[j * p.tile_stride]);
  }
  sm[0][sl][lr] = m;
  __syncthreads();
#pragma unroll
  for (int n = SLICES / 2; n > 0; n /= 2) {
    if (sl < n) sm[0][sl][lr] = fmaxf(sm[0][sl][lr], sm[0][sl + n][lr]);
    __syncthreads();
  }
  const float top = sm[0][0][lr];
  __syncthreads();
  float S = 0.f, U = 0.f;
  if (live) {
#pragma unroll 4
    for (int j = sl; j < p.n_vt; j += SLICES) {
      const float dm = pm[j * p.tile_stride] - top;
      const float a = __expf(dm), s = ps[j * p.tile_stride];
      S += s * a;
      if constexpr (ENT) U += a * (p.part_u[row * p.token_stride + j * p.tile_stride] + dm * s);
    }
  }
  sm[0][sl][lr] = S;
  sm[1][sl][lr] = U;
  __syncthreads();
#pragma unroll
  for (int n = SLICES / 2; n > 0; n /= 2) {
    if (sl < n) {
      sm[0][sl][lr] += sm[0][sl + n][lr];
      if constexpr (ENT) sm[1][sl][lr] += sm[1][sl + n][lr];
    }
    __syncthreads();
  }
  if (sl != 0 || !live) return;
  const float logS = log_sum(sm[0][0][lr]);
  const int64_t t = p.targets[row];
  const bool valid = t != p.ignore_index && t >= 0 && t < p.V;
  float z = zt[lr];
  if constexpr (ROWS == 1) {
#pragma unroll
    for (int k = 1; k < WAVES; ++k) z += zt[k];
  }
  p.lse[row] = top + logS;
  p.logprob[row] = valid ? at_most_zero(z - (top + logS)) : 0.f;
  if constexpr (ENT) p.entropy[row] = valid ? at_least_zero(logS - sm[1][0][lr] / sm[0][0][lr]) : 0.f;
}

}  // namespace

// Fewer vocabulary rows a workgroup, with the waves sharing K instead, where 128 (and 64
// tokens) would leave less than one and a half workgroups a compute unit, as far as the staged
// tokens fit.  Of the whole call, for the order of summation.  Logits in us by this rule and with
// 128 rows throughout: 1 x 4096 x 8000 6.2 and 8.9, 32 x 4096 x 8000 10.2 and 12.1, 128 x 4096 x
// 8000 11.0 and 13.5; past a vocabulary of about 16000, where one workgroup a unit runs at a
// time, 128 rows are the faster ones: 32 x 4096 x 24000 18.3 and 13.3, 64 x 4096 x 40000 28.7 and
// 26.3, 32 x 2048 x 24000 15.0 and 10.4.
int mx_stream_rows(long M, int V) {
  const int64_t n_mt = (M + 63) / 64;
  if ((V + 127) / 128 * n_mt >= 384) return 128;
  if (M > 32 || (V + 63) / 64 >= 384) return 64;
  return 32;
}

hipError_t launch_mx_stream_logits(const MxLogitsArgs& a, hipStream_t s) {
  const int rows = mx_stream_rows(a.call_M, a.V);
  const unsigned g = (unsigned)(((int64_t)a.V + rows - 1) / rows);
  with_tokens(a.M, a.V, a.X != nullptr, rows, [&](auto cfg) {
    using C = decltype(cfg);
    const unsigned n = g * (unsigned)((a.M + 32 * C::TB - 1) / (32 * C::TB));
    if (a.out_dtype == kBf16) mx_stream_logits_kernel<C, Bf16><<<n, 256, 0, s>>>(a);
    else mx_stream_logits_kernel<C, F32><<<n, 256, 0, s>>>(a);
  });
  return hipGetLastError();
}

hipError_t launch_mx_stream_fwd(const MxFwdArgs& a, hipStream_t s) {
  with_tokens(a.M, a.V, a.X != nullptr, mx_stream_rows(a.call_M, a.V), [&](auto cfg) {
    using C = decltype(cfg);
    const unsigned n = (unsigned)a.n_vt * (unsigned)((a.M + 32 * C::TB - 1) / (32 * C::TB));
    if (a.part_u) mx_stream_fwd_kernel<C, true><<<n, 256, 0, s>>>(a);
    else mx_stream_fwd_kernel<C, false><<<n, 256, 0, s>>>(a);
  });
  return hipGetLastError();
}

template <int ROWS>
static void merge_rows(const MxFwdArgs& a, hipStream_t s) {
  const unsigned g = (unsigned)(((long)a.M + ROWS - 1) / ROWS);
  if (a.part_u) mx_merge_kernel<ROWS, true><<<g, MERGE_THREADS, 0, s>>>(a);
  else mx_merge_kernel<ROWS, false><<<g, MERGE_THREADS, 0, s>>>(a);
}

// The whole call's tokens choose the kernel, for its order of summation: waves of any height
// then give the same bits.
hipError_t launch_mx_merge(const MxFwdArgs& a, hipStream_t s) {
  if (a.tile_stride == 1) merge_rows<1>(a, s);
  else if (a.call_M <= 1024) merge_rows<4>(a, s);
  else merge_rows<16>(a, s);
  return hipGetLastError();
}

}  // namespace flce
