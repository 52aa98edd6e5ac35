// Log-probs of given tokens, entropy and the largest alternatives from a matrix of logits, and
// their gradient (gfx950).
//
//   m = max_v x_v,  S = sum_v exp(scale (x_v - m)),  logp_v = scale (x_v - m) - log S
//   lse = scale m + log S,  entropy = log S - sum_v exp(scale (x_v - m)) scale (x_v - m) / S
//   dx_v = scale (sum_j g_j (1[v = t_j] - p_v) - b p_v (logp_v + entropy) + c p_v)
//          g, b, c: gradients of the log-probs, the entropy and lse
//
// Both are bound by memory: the logits are read once, with the running maximum, the sums and
// the alternatives of a row kept on the way, and the gradient reads them once more and writes
// as much.  A workgroup takes a row, or a piece of it where there are few rows; the pieces
// meet in a second kernel.
//
// Alternatives: candidates above a running threshold go to LDS with their index.  The first step
// (64 bytes a thread: 8192 bf16 logits, 4096 fp32) sets it: the k-th largest of the 256 threads'
// own maxima is at most the k-th largest of all (k different elements reach it), and about k
// elements lie above it.  When candidates pile up, the k-th largest of them (found bit by bit, the
// counts by ballots) becomes the threshold and the others go.  So of a row of independent logits
// some 5 k ever reach LDS; rows in ascending order reach it whole, in steps that fit.  Order is
// that of the logits, equal ones by their index; the order in which candidates arrive changes
// nothing.
//
// Measured (us, calls among others): 4096 x 128256 bf16 without alternatives 184 (5.7 TB/s; the
// entropy adds 4), with 20 of them 232 (242 in a trace, where a launch waits for the one before);
// 2048 x 128256 fp32 with 20 187; 257 x 50257 fp32 without 16, with 8 25; 4 x 128256 fp32 without 6.2,
// with 5 13, in a trace 8.2 for the pieces and 5.3 for the joining kernel.  What the alternatives cost
// is a row's fixed part, in which only the next step's loads are in flight: the first threshold, two
// barriers a step, the last thinning (4096 x 32768 bf16: 49 without, 74 with 5, 123 with 50).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_internal.h"
#include "mx_device.h"
#include "tile_device.h"

namespace flce {

namespace {

constexpr int T = 256;              // threads of a workgroup
constexpr int VEC_STEP = 8 * T;     // logits of one vector (8 logits) of every thread
// Vectors that a thread holds at once: 64 bytes.
template <class TX>
constexpr int NV = sizeof(typename TX::mem) == 2 ? 4 : 2;
template <class TX>
constexpr int STEP = NV<TX> * VEC_STEP;
constexpr int CAP = 2048;           // candidates in LDS
constexpr int CROWDED = 32;         // more than this and 3 k are thinned out
constexpr int SPARE = 64;           // equal logits kept beyond k without a look at their index
constexpr float LOWEST = -3.402823466e38f;
static_assert(CAP >= CROWDED + 3 * kMaxTop && CAP >= kMaxTop + SPARE + VEC_STEP / 2, "half a vector of every thread fits after thinning");

// Floats ordered as whole numbers.  -0 is 0, and a NaN ranks with -inf.
constexpr uint32_t KEY_NONE = 0x007fffffu;  // -inf
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  const uint32_t k = u & 0x80000000u ? ~u : u | 0x80000000u;
  return x > -INFINITY ? k : KEY_NONE;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
// A float that everything of at least this key exceeds, and nothing else does (-inf: all numbers
// exceed it; below 0 comes the first negative number, not -0).
__device__ __forceinline__ float below(uint32_t k) {
  return k <= KEY_NONE + 1 ? -INFINITY : value_of(k == 0x80000000u ? k - 2 : k - 1);
}

// A candidate: its logit's key above the complement of its index, so that the larger of two comes
// first.
typedef unsigned long long Candidate;
__device__ __forceinline__ Candidate candidate(float x, int index) {
  return (Candidate)key_of(x) << 32 | ~(uint32_t)index;
}
__device__ __forceinline__ uint32_t key_in(Candidate c) { return (uint32_t)(c >> 32); }
__device__ __forceinline__ uint32_t index_in(Candidate c) { return ~(uint32_t)c; }

// Candidates of a row, and what the waves tell each other.
struct Shared {
  Candidate cand[CAP];
  uint32_t lane_key[T];
  int count;
  float threshold;
  float red[3][T / 64];
};

__device__ __forceinline__ int count_of(bool b) { return __popcll(__ballot(b)); }

// The largest t with count(t) >= k, for a count that falls with t, where the answer shares the
// bits above `bits` with `prefix`; found early where the count is k exactly.
template <class Count>
__device__ __forceinline__ uint32_t kth(uint32_t prefix, int bits, int k, Count count) {
  uint32_t t = prefix;
  for (int b = bits - 1; b >= 0; --b) {
    const uint32_t c = t | (1u << b);
    const int n = count(c);
    if (n >= k) t = c;
    if (n == k) break;
  }
  return t;
}
// Bits in which values between lo and hi may differ, and the rest of them.
__device__ __forceinline__ int open_bits(uint32_t lo, uint32_t hi) {
  return lo == hi ? 0 : 32 - __clz((int)(lo ^ hi));
}
__device__ __forceinline__ uint32_t closed(uint32_t lo, int bits) { return bits >= 32 ? 0u : lo >> bits << bits; }

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint32_t w = (uint32_t)__shfl_xor((int)v, o);
    v = v > w ? v : w;
  }
  return v;
}
__device__ __forceinline__ uint32_t wave_min(uint32_t v) { return ~wave_max(~v); }

// Wave 0: keep the k largest of sh.count > k candidates, and up to SPARE more that equal the
// last of them; the threshold becomes that one's logit.  Candidates that come later have larger
// indexes, so only larger logits can displace what is kept.  Up to 256 keys (the usual case) stay
// in registers while the bits of the k-th largest are found.
__device__ __forceinline__ void thin_out(Shared& sh, int k) {
  const int lane = threadIdx.x & 63, n = min(sh.count, CAP);
  uint32_t held[4], lo = ~0u, hi = 0u;
#pragma unroll
  for (int w = 0; w < 4; ++w) held[w] = 64 * w + lane < n ? key_in(sh.cand[64 * w + lane]) : 0u;
  for (int i = lane; i < n; i += 64) {
    lo = min(lo, key_in(sh.cand[i]));
    hi = max(hi, key_in(sh.cand[i]));
  }
  lo = wave_min(lo);
  hi = wave_max(hi);
  const int bits = open_bits(lo, hi);
  // (keys are not 0, and neither is what they are compared with)
  const uint32_t t = kth(closed(lo, bits), bits, k, [&](uint32_t c) {
    int s = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) s += count_of(held[w] >= c);
    for (int i = 256 + lane; i < n + lane; i += 64) s += count_of(i < n && key_in(sh.cand[i]) >= c);
    return s;
  });
  // (t may lie between two candidates: the threshold is the least one at or above it)
  int above = 0, equal = 0;
  uint32_t least = ~0u;
  for (int i = lane; i < n; i += 64) {
    const uint32_t key = key_in(sh.cand[i]);
    if (key >= t) least = min(least, key);
  }
  least = wave_min(least);
  for (int i = lane; i < n + lane; i += 64) {
    const uint32_t key = i < n ? key_in(sh.cand[i]) : 0u;
    above += count_of(key > least);
    equal += count_of(key == least);
  }
  uint32_t last = 0u;  // the smallest complement of an index kept among equal ones
  if (above + equal > k + SPARE) {
    last = kth(0u, 32, k - above, [&](uint32_t c) {
      int s = 0;
      for (int i = lane; i < n + lane; i += 64)
        s += count_of(i < n && key_in(sh.cand[i]) == least && (uint32_t)sh.cand[i] >= c);
      return s;
    });
  }
  const Candidate cut = (Candidate)least << 32 | last;
  // compact in place: what a step reads lies at or behind what it writes
  int kept = 0;
  for (int i = lane; i < n + lane; i += 64) {
    const Candidate c = i < n ? sh.cand[i] : 0ull;
    const unsigned long long mask = __ballot(c >= cut);
    if (c >= cut) sh.cand[kept + __popcll(mask & ((1ull << lane) - 1ull))] = c;
    kept += __popcll(mask);
  }
  if (lane == 0) {
    sh.count = kept;
    sh.threshold = value_of(least);
  }
}

// Every thread: thin out where there are more candidates than `most`.  The count is read between
// two barriers, so that all threads decide alike.
__device__ __forceinline__ void settle(Shared& sh, int k, int most) {
  __syncthreads();
  const int n = sh.count;
  __syncthreads();
  if (n > most && n > k) {
    if (threadIdx.x < 64) thin_out(sh, k);
    __syncthreads();
  }
}

// Running maximum and sums of one thread: s = sum 2^d, u = sum 2^d d, d = c (x - m).
template <bool ENT>
struct Sums {
  float m = LOWEST, s = 0.f, u = 0.f;
  __device__ __forceinline__ void raise(float to, float c) {
    // (bounded, so that nothing of a sum that is still 0 becomes 0 times infinity)
    const float d = fmaxf((m - to) * c, -1e30f), r = __builtin_amdgcn_exp2f(d);
    if constexpr (ENT) u = r * fmaf(d, s, u);
    s *= r;
    m = to;
  }
  __device__ __forceinline__ void add(const float (&x)[8], float top, float c) {
    if (top > m) raise(top, c);
    float e[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = (x[i] - m) * c;
      e[i] = __builtin_amdgcn_exp2f(d);
      // (a masked logit: 0 times its bound)
      if constexpr (ENT) w[i] = e[i] * fmaxf(d, -1e30f);
    }
    s += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    if constexpr (ENT) u += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
  }
};

// Their largest, or a NaN where one of them is a signaling one (v_max3_f32 issued directly: fmaxf
// quiets each input first).
__device__ __forceinline__ float max8(const float (&x)[8]) {
  return max3_run<false>(max3_run<false>(max3_run<false>(max_raw(x[0], x[1]), x[2], x[3]), x[4], x[5]), x[6], x[7]);
}

// (m, s, u) of the workgroup from those of its threads, in every thread.
template <bool ENT>
__device__ __forceinline__ void join(Sums<ENT>& a, Shared& sh, float c) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float m = a.m;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if (lane == 0) sh.red[0][wave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 64; ++w) m = fmaxf(m, sh.red[0][w]);
  a.raise(m, c);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    a.s += __shfl_xor(a.s, o);
    if constexpr (ENT) a.u += __shfl_xor(a.u, o);
  }
  if (lane == 0) {
    sh.red[1][wave] = a.s;
    if constexpr (ENT) sh.red[2][wave] = a.u;
  }
  __syncthreads();
  a.s = sh.red[1][0];
  a.u = ENT ? sh.red[2][0] : 0.f;
#pragma unroll
  for (int w = 1; w < T / 64; ++w) {
    a.s += sh.red[1][w];
    if constexpr (ENT) a.u += sh.red[2][w];
  }
}

// The place of candidate c among the n (n is small: the last thinning left at most k + SPARE).
__device__ __forceinline__ int rank_of(const Shared& sh, Candidate c, int n) {
  int r = 0, j = 0;
  for (; j + 8 <= n; j += 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r += sh.cand[j + i] > c;
  }
  for (; j < n; ++j) r += sh.cand[j] > c;
  return r;
}

// A row's results from its sums and, in LDS, its candidates.
template <class TX, bool TOP>
__device__ __forceinline__ void finish_row(const TokenLogprobArgs& p, long row, float m, float s, float u,
                                           Shared& sh) {
  const typename TX::mem* x = static_cast<const typename TX::mem*>(p.logits) + row * p.ldl;
  const float nan = __uint_as_float(0x7fc00000u);
  // s: 0 where every logit is masked, a NaN where one is an infinity or a NaN
  const bool none = s == 0.f, bad = !(s >= 0.f) || m == INFINITY;
  const float logs = bad ? nan : none ? 0.f : logf(s);
  const float top = bad ? nan : none ? -INFINITY : m;
  auto logp = [&](float v) { return bad ? nan : none ? -INFINITY : at_most_zero(p.scale * (v - top) - logs); };
  if (threadIdx.x == 0) {
    p.stats[2 * row] = top;
    p.stats[2 * row + 1] = logs;
    p.lse[row] = fmaf(p.scale, top, logs);
    if (p.entropy) p.entropy[row] = bad ? nan : none ? 0.f : at_least_zero(logs - u * LN2 / s);
  }
  for (int j = threadIdx.x; j < p.n_tokens; j += T) {
    const int64_t t = p.tokens[row * p.n_tokens + j];
    const bool valid = t != p.ignore_index && t >= 0 && t < p.V;
    p.logprob[row * p.n_tokens + j] = valid ? logp(TX::to_f32(x[t])) : 0.f;
  }
  if constexpr (TOP) {
    const int n = sh.count, k = p.n_top;
    for (int i = threadIdx.x; i < n; i += T) {
      const Candidate own = sh.cand[i];
      const int r = rank_of(sh, own, n);
      if (r < k) {
        p.top_ids[row * k + r] = (int64_t)index_in(own);
        p.top_logprob[row * k + r] = logp(value_of(key_in(own)));
      }
    }
    // fewer than k logits above -inf: the first of the others follow.  Fewer than k of the first
    // 2 k logits are above it, so those hold enough (k <= V)
    if (n < k && threadIdx.x < 64) {
      int at = n;
      for (int v0 = 0; v0 < min(2 * k, p.V); v0 += 64) {
        const int v = v0 + (int)threadIdx.x;
        const bool masked = v < p.V && !(TX::to_f32(x[v < p.V ? v : 0]) > -INFINITY);
        const unsigned long long mask = __ballot(masked);
        const int r = at + __popcll(mask & ((1ull << threadIdx.x) - 1ull));
        if (masked && r < k) {
          p.top_ids[row * k + r] = v;
          p.top_logprob[row * k + r] = bad ? nan : -INFINITY;
        }
        at += __popcll(mask);
      }
    }
  }
}

// 8 consecutive logits as they lie in memory, at any alignment of an element.
template <class TX>
struct Raw8 {
  static constexpr bool HALF = sizeof(typename TX::mem) == 2;
  static constexpr int N = HALF ? 1 : 2;
  u32x4_t u[N];
  __device__ __forceinline__ void load(const typename TX::mem* x) {
    if constexpr (HALF) {
      u[0] = *reinterpret_cast<const u32x4_a2*>(x);
    } else {
      u[0] = *reinterpret_cast<const u32x4_a4*>(x);
      u[1] = *reinterpret_cast<const u32x4_a4*>(x + 4);
    }
  }
  // The first n of them, then -inf.
  __device__ __forceinline__ void load_part(const typename TX::mem* x, int n) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t none = HALF ? 0xff80ff80u : 0xff800000u;
      u[k] = u32x4_t{none, none, none, none};
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (HALF) u[0][i / 2] = i & 1 ? (u[0][i / 2] & 0xffffu) | (uint32_t)x[i] << 16 : (u[0][i / 2] & 0xffff0000u) | x[i];
        else u[i / 4][i & 3] = __float_as_uint(x[i]);
      }
  }
  __device__ __forceinline__ void value(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (HALF) v[i] = i & 1 ? bf16_hi(u[0][i / 2]) : bf16_lo(u[0][i / 2]);
      else v[i] = __uint_as_float(u[i / 4][i & 3]);
    }
  }
};

// The logits of [base, v1) of the next N vectors of every thread.
template <class TX, int N>
__device__ __forceinline__ void load_step(Raw8<TX> (&raw)[N], const typename TX::mem* x, int base, int v1) {
  const int col = base + 8 * (int)threadIdx.x;
  if (base + N * VEC_STEP <= v1) {
#pragma unroll
    for (int j = 0; j < N; ++j) raw[j].load(x + col + j * VEC_STEP);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int c = col + j * VEC_STEP;
      if (c + 8 <= v1) raw[j].load(x + c);
      else raw[j].load_part(x + c, v1 - c);
    }
  }
}

__device__ __forceinline__ void offer(Shared& sh, float value, float threshold, int col) {
  if (value > threshold) {
    const int at = atomicAdd(&sh.count, 1);
    if (at < CAP) sh.cand[at] = candidate(value, col);
  }
}

// The candidates of one step do not fit: they are offered again in halves of a vector, thinned
// out after each.  Indexes do not ascend from one half to the next, so the halves keep the
// threshold of the steps before them, and offer what equals a later one too.
template <class TX>
__device__ __forceinline__ void offer_in_parts(Shared& sh, const typename TX::mem* x, int base, int v1, int held,
                                               float threshold, int k) {
  if (threadIdx.x == 0) sh.count = held;
  __syncthreads();
  settle(sh, k, k + SPARE);
  if (held > k + SPARE) threshold = sh.threshold;
#pragma unroll 1
  for (int h = 0; h < 2 * NV<TX>; ++h) {
    const int col = base + (h >> 1) * VEC_STEP + 8 * (int)threadIdx.x + 4 * (h & 1);
#pragma unroll 1
    for (int i = 0; i < 4; ++i)
      if (col + i < v1) offer(sh, TX::to_f32(x[col + i]), threshold, col + i);
    settle(sh, k, k + SPARE);
  }
}

// The next step's loads are in flight under the work on this one.  With alternatives in bf16 the
// registers of five workgroups a unit are too few (10 a thread go to memory without the entropy, 6
// with it; of four 2 and none), but five overlap more rows' fixed parts: neither is better throughout,
// long rows with few alternatives want four, short ones with many five.  4096 rows of bf16, us with four
// and five (six are 10 to 80% slower):
//            without the entropy           with it
//   V        k = 5     20        50        5         20        50
//   128256   208, 235  234, 243  284, 266  212, 229  249, 242  300, 275
//   32768    74, 76    99, 93    123, 114  76, 75    102, 95   126, 116
// Four without the entropy and five with it are the better side at 128256 with 20.  Without
// alternatives both take the same time (182, 188; 49, 51); fp32 at 2048 x 128256 with 20 takes 186, 195
// and 188, 190.
template <class TX, bool ENT, bool TOP>
__global__ __launch_bounds__(T, ENT ? 5 : 4) void token_logprob_kernel(TokenLogprobArgs p) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, k = p.n_top, crowded = CROWDED + 3 * k;
  const float c = p.scale * LOG2E;
  const long items = p.M * p.parts;
  for (long item = blockIdx.x; item < items; item += gridDim.x) {
    const long row = item / p.parts;
    const int part = (int)(item - row * p.parts);
    const int v0 = part * p.part_len, v1 = min(p.V, v0 + p.part_len);
    const typename TX::mem* x = static_cast<const typename TX::mem*>(p.logits) + row * p.ldl;
    Sums<ENT> sums;
    float threshold = -INFINITY;
    int held = 0;  // candidates in LDS
    if constexpr (TOP) {
      if (tid == 0) sh.count = 0;
    }
    Raw8<TX> raw[NV<TX>], next[NV<TX>];
    load_step<TX>(next, x, v0, v1);
    for (int base = v0; base < v1; base += STEP<TX>) {
#pragma unroll
      for (int j = 0; j < NV<TX>; ++j) raw[j] = next[j];
      if (base + STEP<TX> < v1) load_step<TX>(next, x, base + STEP<TX>, v1);
      float top[NV<TX>];
#pragma unroll
      for (int j = 0; j < NV<TX>; ++j) {
        float v[8];
        raw[j].value(v);
        top[j] = max8(v);
        sums.add(v, top[j], c);
      }
      if constexpr (TOP) {
        if (base == v0) {
          float most = top[0];
#pragma unroll
          for (int j = 1; j < NV<TX>; ++j) most = fmaxf(most, top[j]);
          sh.lane_key[tid] = key_of(most);
          __syncthreads();
          uint32_t mine[T / 64], hi = 0u, lo = ~0u;
#pragma unroll
          for (int w = 0; w < T / 64; ++w) {
            mine[w] = sh.lane_key[64 * w + (tid & 63)];
            hi = max(hi, mine[w]);
            lo = min(lo, mine[w]);
          }
          hi = wave_max(hi);
          lo = wave_min(lo);
          // (every wave for itself: the same answer)
          const int bits = open_bits(lo, hi);
          threshold = below(kth(closed(lo, bits), bits, k, [&](uint32_t cand) {
            int n = 0;
#pragma unroll
            for (int w = 0; w < T / 64; ++w) n += count_of(mine[w] >= cand);
            return n;
          }));
        }
        // (a thread's candidates of the step take their places with one atomic)
        uint32_t hits = 0u;
#pragma unroll
        for (int j = 0; j < NV<TX>; ++j)
          if (!(top[j] <= threshold)) {
            float v[8];
            raw[j].value(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) hits |= v[i] > threshold ? 1u << (8 * j + i) : 0u;
          }
        if (hits) {
          int at = atomicAdd(&sh.count, __popc(hits));
#pragma unroll
          for (int j = 0; j < NV<TX>; ++j)
            if (hits >> (8 * j) & 255u) {
              float v[8];
              raw[j].value(v);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (hits >> (8 * j + i) & 1u) {
                  if (at < CAP) sh.cand[at] = candidate(v[i], base + j * VEC_STEP + 8 * tid + i);
                  ++at;
                }
            }
        }
        __syncthreads();
        const int now = sh.count;  // (between barriers: the same for every thread)
        __syncthreads();
        if (now <= crowded) {
          held = now;
        } else {
          if (now <= CAP) {
            if (tid < 64) thin_out(sh, k);
            __syncthreads();
          } else {
            offer_in_parts<TX>(sh, x, base, v1, held, threshold, k);
          }
          threshold = sh.threshold;
          held = sh.count;
          __syncthreads();
        }
      }
    }
    join<ENT>(sums, sh, c);
    if constexpr (TOP) settle(sh, k, k + SPARE);
    if (p.parts == 1) {
      finish_row<TX, TOP>(p, row, sums.m, sums.s, sums.u, sh);
    } else {
      if (tid == 0) {
        float* to = p.part_sums + 3 * item;
        to[0] = sums.m;
        to[1] = sums.s;
        to[2] = sums.u;
      }
      if constexpr (TOP) {
        const int n = sh.count;
        Candidate* to = p.part_top + item * k;
        for (int i = tid; i < n; i += T) {
          const Candidate own = sh.cand[i];
          const int r = rank_of(sh, own, n);
          if (r < k) to[r] = own;
        }
        for (int r = n + tid; r < k; r += T) to[r] = 0ull;
      }
    }
    __syncthreads();
  }
}

// The pieces of a row: their sums rescaled to the largest maximum, their candidates together.  A
// piece's list is in order, so where q pieces reach x with their a-th entry, a q entries are x or
// more: with a q >= k the q-th largest of the a-th entries bounds what can count, and leaves little
// more than k of the lists' entries.  All loads go out at once: this kernel is a chain of waits.
template <class TX, bool TOP>
__global__ __launch_bounds__(T) void token_logprob_join_kernel(TokenLogprobArgs p) {
  __shared__ Shared sh;
  constexpr int HELD = CAP / T;  // entries of a thread
  const int tid = threadIdx.x, k = p.n_top;
  const float c = p.scale * LOG2E;
  for (long row = blockIdx.x; row < p.M; row += gridDim.x) {
    // a piece a thread (there are at most 128)
    const bool mine = tid < p.parts;
    const float* part = p.part_sums + 3 * (row * p.parts + (mine ? tid : 0));
    Sums<true> sums;
    sums.m = mine ? part[0] : LOWEST;
    sums.s = mine ? part[1] : 0.f;
    sums.u = mine ? part[2] : 0.f;
    const int n = TOP ? p.parts * k : 0;  // at most CAP
    const Candidate* from = p.part_top + row * n;
    Candidate entry[HELD];
    if constexpr (TOP) {
#pragma unroll
      for (int i = 0; i < HELD; ++i) entry[i] = tid + i * T < n ? from[tid + i * T] : 0ull;
      const int a = (k + p.parts - 1) / p.parts;
      sh.lane_key[tid] = mine ? key_in(from[tid * k + a - 1]) : 0u;
      if (tid == 0) sh.count = 0;
    }
    join<true>(sums, sh, c);
    if constexpr (TOP) {
      const int a = (k + p.parts - 1) / p.parts, q = (k + a - 1) / a, lane = tid & 63;
      const uint32_t one = sh.lane_key[lane], two = sh.lane_key[64 + lane];
      const int bits = open_bits(0u, wave_max(max(one, two)));
      // (an entry of no candidate is 0; where fewer than q pieces have an a-th one, all count)
      const uint32_t least =
          max(1u, kth(0u, bits, q, [&](uint32_t cand) { return count_of(one >= cand) + count_of(two >= cand); }));
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (key_in(entry[i]) >= least) sh.cand[atomicAdd(&sh.count, 1)] = entry[i];
      settle(sh, k, k + SPARE);
    }
    finish_row<TX, TOP>(p, row, sums.m, sums.s, sums.u, sh);
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// The gradient: a workgroup takes a piece of a row.  What the given tokens add is computed first
// (from the logits, so dlogits may be the logits' own memory) and written over the rest after a
// barrier; several entries of one token are added in their order.
//
// Bound by memory: 4096 x 32768 bf16 with one token 97 us (5.5 TB/s), 513 x 50257 fp32 with 64 48
// (4.3 TB/s), 4096 x 50257 fp32 297 (5.5 TB/s).
constexpr int LIST = kMaxTokens + kMaxTop;
static_assert(LIST % 8 == 0, "groups of 8");
constexpr int GRAD_NV = 4, GRAD_STEP = GRAD_NV * VEC_STEP;

struct GradShared {
  int id[LIST];     // the entry's token, -1 outside this piece
  float g[LIST];
  int at[LIST];     // where the entry's thread writes `value`, -1: nowhere
  float value[LIST];
  float red[T / 64];
  int any[T / 64];
};

template <class TX>
__global__ __launch_bounds__(T) void token_logprob_grad_kernel(TokenLogprobGradArgs p, int pieces) {
  __shared__ GradShared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int L = p.n_tokens + p.n_top;
  const long items = p.M * pieces;
  for (long item = blockIdx.x; item < items; item += gridDim.x) {
    const long row = item / pieces;
    const int v0 = (int)(item - row * pieces) * GRAD_STEP, v1 = min(p.V, v0 + GRAD_STEP);
    const typename TX::mem* x = static_cast<const typename TX::mem*>(p.logits) + row * p.ldl;
    typename TX::mem* dx = static_cast<typename TX::mem*>(p.dlogits) + row * p.ldd;
    Raw8<TX> raw[GRAD_NV];
    load_step<TX>(raw, x, v0, v1);
    const float top = p.stats[2 * row], logs = p.stats[2 * row + 1];
    const float b = p.grad_entropy ? p.grad_entropy[row] : 0.f, ent = p.grad_entropy ? p.entropy[row] : 0.f;
    const float of_lse = p.grad_lse ? p.grad_lse[row] : 0.f;

    // the list of (token, gradient): their sum, and those of this piece
    float sum = 0.f;
    bool any = false;
    if (tid < 8 && L + tid < LIST) {
      sh.id[L + tid] = -1;
      sh.g[L + tid] = 0.f;
    }
    for (int j = tid; j < L; j += T) {
      const bool given = j < p.n_tokens;
      const long at = given ? row * p.n_tokens + j : row * p.n_top + (j - p.n_tokens);
      const int64_t t = given ? p.tokens[at] : p.top_ids[at];
      const bool valid = !(given && t == p.ignore_index) && t >= 0 && t < p.V;
      const float g = valid ? (given ? p.grad_logprob : p.grad_top)[at] : 0.f;
      sum += g;
      any |= valid;
      sh.id[j] = valid && t >= v0 && t < v1 ? (int)t : -1;
      sh.g[j] = g;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    const bool any_wave = __any(any);
    if (lane == 0) {
      sh.red[wave] = sum;
      sh.any[wave] = any_wave;
    }
    __syncthreads();
    sum = sh.red[0];
    any = sh.any[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) {
      sum += sh.red[w];
      any |= sh.any[w] != 0;
    }
    // a row that nothing is asked of, or in which everything is masked, has no gradient
    const bool zero = (!any && b == 0.f && of_lse == 0.f) || top == -INFINITY;
    // dx = scale (g + p_v (k0 - b logp_v)), 0 where p_v is 0 however large its factor.  scale comes last:
    // scale b times a log-prob of some hundred may pass fp32's range where dx does not.
    const float k0 = of_lse - fmaf(b, ent, sum);
    auto slope = [&](float v) {
      const float lp = fmaf(p.scale, v - top, -logs), pv = __builtin_amdgcn_exp2f(lp * LOG2E);
      return pv > 0.f ? pv * fmaf(-b, lp, k0) : 0.f;
    };
    // (a NaN in the row's statistics or gradients has to reach every element: the choice would drop it)
    const float add_nan = zero ? 0.f : 0.f * (top + logs) + (k0 != k0 ? k0 : 0.f);

    for (int j = tid; j < L; j += T) {
      const int id = zero ? -1 : sh.id[j];
      int first = -1;  // the first entry of this token
      float g = 0.f;
      if (id >= 0) {
        first = j;
        // (whole groups of 8: the list is padded with entries of no token)
        for (int i0 = 0; i0 < L; i0 += 8)
#pragma unroll
          for (int i = i0; i < i0 + 8; ++i) {
            const bool same = sh.id[i] == id;
            first = same ? min(first, i) : first;
            g += same ? sh.g[i] : 0.f;
          }
      }
      sh.at[j] = first == j ? id : -1;
      if (first == j) sh.value[j] = p.scale * (g + slope(TX::to_f32(x[id]))) + add_nan;
    }
    // (every read of these logits by hand is done before any is overwritten)
    wait_vmcnt<0>();
    __syncthreads();
#pragma unroll
    for (int j = 0; j < GRAD_NV; ++j) {
      const int col = v0 + j * VEC_STEP + 8 * tid;
      float v[8];
      raw[j].value(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = zero ? 0.f : fmaf(p.scale, slope(v[i]), add_nan);
      if (col < v1) store8<TX, false>(dx, col, p.V, v);
    }
    wait_vmcnt<0>();
    __syncthreads();
    for (int j = tid; j < L; j += T)
      if (sh.at[j] >= 0) dx[sh.at[j]] = TX::from_f32(sh.value[j]);
  }
}

template <class TX, bool ENT>
void run_parts(const TokenLogprobArgs& a, unsigned grid, hipStream_t s) {
  if (a.n_top) token_logprob_kernel<TX, ENT, true><<<grid, T, 0, s>>>(a);
  else token_logprob_kernel<TX, ENT, false><<<grid, T, 0, s>>>(a);
}
template <class TX>
void run(const TokenLogprobArgs& a, hipStream_t s) {
  const long items = a.M * a.parts, most = 1 << 22;
  const unsigned grid = (unsigned)(items < most ? items : most);
  if (a.entropy) run_parts<TX, true>(a, grid, s);
  else run_parts<TX, false>(a, grid, s);
  if (a.parts > 1) {
    const unsigned rows = (unsigned)(a.M < most ? a.M : most);
    if (a.n_top) token_logprob_join_kernel<TX, true><<<rows, T, 0, s>>>(a);
    else token_logprob_join_kernel<TX, false><<<rows, T, 0, s>>>(a);
  }
}

}  // namespace

void token_logprob_split(int64_t M, int64_t V, int n_top, int* parts, int* part_len) {
  const int64_t pieces = (V + VEC_STEP - 1) / VEC_STEP;
  int64_t want = M >= 1024 || M < 1 ? 1 : 1024 / M;
  if (want > 128) want = 128;
  if (n_top && want > CAP / n_top) want = CAP / n_top;
  if (want > pieces) want = pieces;
  const int64_t each = (pieces + want - 1) / want;
  *part_len = int(each * VEC_STEP);
  *parts = int((pieces + each - 1) / each);
}

hipError_t launch_token_logprobs(const TokenLogprobArgs& a, int dtype, hipStream_t s) {
  if (dtype == kF32) run<F32>(a, s);
  else run<Bf16>(a, s);
  return hipGetLastError();
}

hipError_t launch_token_logprobs_grad(const TokenLogprobGradArgs& a, int dtype, hipStream_t s) {
  const int pieces = (a.V + GRAD_STEP - 1) / GRAD_STEP;
  const long items = a.M * pieces, most = 1 << 22;
  const unsigned grid = (unsigned)(items < most ? items : most);
  if (dtype == kF32) token_logprob_grad_kernel<F32><<<grid, T, 0, s>>>(a, pieces);
  else token_logprob_grad_kernel<Bf16><<<grid, T, 0, s>>>(a, pieces);
  return hipGetLastError();
}

}  // namespace flce
