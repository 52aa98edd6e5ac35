// Internal interface between the libflce host code and the kernels of the residual block in
// front of the head (matrix product with an epilogue, dropout) and of the log-probs read off a
// matrix of logits.  Not installed; not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "flce_internal.h"

namespace flce {

// ---------------------------------------------------------------- dropout
struct DropoutArgs {
  const void* x;
  long ldx;                 // elements between rows
  const void* residual;     // nullptr: none
  long ldr;
  void* y;
  long ldy;
  long M;
  int H;
  uint32_t threshold;       // an element is dropped where its 16 bits are below it
  float up;                 // 65536 / (65536 - threshold); 0 where nothing is kept
  uint64_t seed;
  const uint64_t* seed_at;  // nullptr: `seed`; else the seed's place in device memory
  uint64_t offset;
};
constexpr int kNoResidual = -1;
// residual_dtype: kNoResidual, kBf16 or kF32.
hipError_t launch_dropout(const DropoutArgs& a, int x_dtype, int residual_dtype, int y_dtype, bool vec,
                          hipStream_t s);

// ---------------------------------------------------------------- log-probs from logits
constexpr int kMaxTop = 128;      // alternatives of a row
constexpr int kMaxTokens = 1024;  // given tokens of a row
struct TokenLogprobArgs {
  const void* logits;
  long ldl;                 // elements between rows
  long M;
  int V;
  const int64_t* tokens;    // [M, n_tokens]
  int n_tokens;
  int64_t ignore_index;
  float scale;
  int n_top;
  float* logprob;           // [M, n_tokens]
  float* lse;               // [M]
  float* entropy;           // [M] or nullptr
  float* stats;             // [M, 2]: the row's largest logit, the log of its shifted sum
  int64_t* top_ids;         // [M, n_top]
  float* top_logprob;       // [M, n_top]
  int parts;                // pieces of a row, a workgroup each
  int part_len;             // elements of a piece
  float* part_sums;         // [M, parts, 3] (parts > 1)
  unsigned long long* part_top;  // [M, parts, n_top]
};
// Pieces a row is split into, and the elements of each.
void token_logprob_split(int64_t M, int64_t V, int n_top, int* parts, int* part_len);
hipError_t launch_token_logprobs(const TokenLogprobArgs& a, int dtype, hipStream_t s);

struct TokenLogprobGradArgs {
  const void* logits;
  long ldl;
  long M;
  int V;
  const int64_t* tokens;    // [M, n_tokens]
  int n_tokens;
  int64_t ignore_index;
  float scale;
  const float* stats;       // [M, 2]
  const float* entropy;     // [M], needed with grad_entropy
  const int64_t* top_ids;   // [M, n_top]
  int n_top;
  const float* grad_logprob;  // [M, n_tokens] or nullptr
  const float* grad_top;      // [M, n_top] or nullptr
  const float* grad_entropy;  // [M] or nullptr
  const float* grad_lse;      // [M] or nullptr
  void* dlogits;
  long ldd;
};
hipError_t launch_token_logprobs_grad(const TokenLogprobGradArgs& a, int dtype, hipStream_t s);

// ---------------------------------------------------------------- matrix product with an epilogue
// Activations: the values of the C ABI's enumeration.
constexpr int kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4;

// What happens to a product before it is stored: out = act(product + bias) + residual.
struct LinearEpilogue {
  const void* bias;        // [N] or nullptr
  int bias_dtype;
  int act;
  const void* residual;    // [M, N] or nullptr
  int residual_dtype;
  long ldr;
  void* out;               // [M, N]
  int out_dtype;
  long ldo;
  uint16_t* pre;           // [M, N] bf16: product + bias, or nullptr
  long ldp;
};

// D[m, n] = sum_k A(m, k) B(n, k).  An operand either has its K contiguous in memory (rows of K)
// or its rows (K rows of M or N elements): X and W in the forward, dpre and W^T in dX, dpre^T and
// X^T in dW.  Either way ld elements lie between the rows of its memory, which are 16-byte aligned,
// and kvalid_* of K exist.
struct LinearProduct {
  const uint16_t* a;
  const uint16_t* b;
  long lda, ldb;
  int M, N, K;
  int kvalid_a, kvalid_b;
};
// Tile and K split of a product: splits > 1 leave fp32 partial products [splits][M][ldpart] in
// the workspace, which a second kernel adds in order.
struct LinearPlan {
  int tile_m, tile_n;
  int splits, k_each;
};
LinearPlan linear_forward_plan(int64_t M, int64_t N, int64_t K);
void linear_backward_plans(int64_t M, int64_t N, int64_t K, LinearPlan* dx, LinearPlan* dw);
int64_t linear_workgroups(const LinearPlan& p, int64_t M, int64_t N);
// Whether a launch can hold the product's workgroups: half of its limit each, as the gradient's has
// two products, and some beside them.
inline bool linear_fits(const LinearPlan& p, int64_t M, int64_t N) {
  return linear_workgroups(p, M, N) <= kMaxWorkgroups / 2 - (1 << 16);
}
inline int64_t linear_part_ld(int64_t N) { return (N + 7) / 8 * 8; }
inline size_t linear_part_bytes(const LinearPlan& p, int64_t M, int64_t N) {
  return p.splits > 1 ? size_t(p.splits) * size_t(M) * size_t(linear_part_ld(N)) * 4 : 0;
}
// The forward's product (both operands with their K contiguous).
hipError_t launch_linear_product(const LinearProduct& a, const LinearPlan& plan, const LinearEpilogue& e,
                                 float* part, hipStream_t s);

// The gradient's products from dpre and the bias gradient from its column sums.
struct LinearBiasSum {
  const float* part;       // [groups][N]
  int groups, N;
  void* dbias;             // nullptr: not wanted
  int dtype;
};
struct LinearGradArgs {
  LinearProduct dx, dw;
  LinearEpilogue out_dx, out_dw;
  LinearPlan plan_dx, plan_dw;
  float* part_dx;
  float* part_dw;
  int n_dx, n_dw;          // workgroups of each (0: not wanted)
  LinearBiasSum bias;
};
hipError_t launch_linear_grad(LinearGradArgs a, hipStream_t s);

// A few rows of X: W streamed past them, up to kLinearDotRows of them by dot products.
constexpr int kLinearFewRows = 32, kLinearDotRows = 2;
bool linear_takes_few(int64_t M, int64_t N, int64_t K);
hipError_t launch_linear_few(const LinearProduct& a, const LinearEpilogue& e, hipStream_t s);

// dpre = dy act'(pre) in bf16, and the column sums of its unrounded values.
struct LinearSlopeArgs {
  const void* dy;
  int dy_dtype;
  long lddy;
  const uint16_t* pre;     // bf16 [M, N], or nullptr without an activation
  long ldp;
  int act;
  long M;
  int N;
  uint16_t* dpre;          // [M, ldd] or nullptr; columns N .. ldd - 1 are written as 0
  long ldd;
  float* part;             // [groups][N] column sums, or nullptr
  int groups;
  bool vec;
};
int linear_slope_groups(int64_t M, int64_t N);
hipError_t launch_linear_slope(const LinearSlopeArgs& a, hipStream_t s);

// dX of up to kLinearFewDx values from dy and pre themselves.
constexpr int kLinearFewDx = 1024;
inline bool linear_takes_few_dx(int64_t M, int64_t K) { return M * K <= kLinearFewDx; }
struct LinearFewDx {
  const void* dy;
  int dy_dtype;
  long lddy;
  const uint16_t* pre;     // bf16 [M, N], or nullptr without an activation
  long ldp;
  int act;
  const uint16_t* w;       // [N, K]
  long ldw;
  int M, N, K;
  uint16_t* dx;            // [M, K]
  long lddx;
  float* part;             // [splits][M][K]
  int each, splits, lanes; // set by the launch: n a workgroup, shares, lanes along a row of W
};
LinearPlan linear_few_dx_plan(int64_t M, int64_t N, int64_t K);
hipError_t launch_linear_few_dx(LinearFewDx a, const LinearPlan& plan, hipStream_t s);

}  // namespace flce
