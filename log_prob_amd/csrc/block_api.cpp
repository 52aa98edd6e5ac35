// C ABI of the residual block in front of the head (matrix product with an epilogue, dropout)
// and of the log-probs read off a matrix of logits.  Every check runs on the host before the
// first HIP call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_util.h"
#include "block_internal.h"
#include "flce.h"
#include "mx_layout.h"

static_assert(FLCE_BF16 == flce::kBf16 && FLCE_FP32 == flce::kF32, "element types");
static_assert(FLCE_ACT_NONE == flce::kActNone && FLCE_ACT_RELU == flce::kActRelu &&
                  FLCE_ACT_GELU == flce::kActGelu && FLCE_ACT_GELU_TANH == flce::kActGeluTanh &&
                  FLCE_ACT_SILU == flce::kActSilu,
              "activations");
static_assert(FLCE_MAX_TOP == flce::kMaxTop && FLCE_MAX_TOKENS == flce::kMaxTokens, "limits of a row");

namespace {

using flce::fail;
using flce::is_aligned;
using flce::ok;

constexpr size_t kAlign = 256;
constexpr int64_t kMaxStride = int64_t(1) << 40;
// Row stride of an operand of the matrix product: a tile's byte offsets stay below 2^31.
constexpr int64_t kMaxOperandStride = int64_t(1) << 21;

bool is_dtype(int d) { return d == FLCE_BF16 || d == FLCE_FP32; }
size_t bytes_of(int d) { return d == FLCE_BF16 ? 2 : 4; }
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

flce_status_t hip_fail(hipError_t e, const char* what) {
  return fail(FLCE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// A matrix whose rows have `cols` elements: row stride and natural alignment.
flce_status_t check_matrix(const char* name, const void* p, int dtype, int64_t ld, int64_t cols) {
  if (!p) return fail(FLCE_ERR_INVALID_VALUE, "%s is NULL", name);
  if (ld < cols)
    return fail(FLCE_ERR_INVALID_VALUE, "%s: row stride %lld is below its %lld columns", name, (long long)ld,
                (long long)cols);
  if (ld > kMaxStride) return fail(FLCE_ERR_UNSUPPORTED, "%s: row stride too large (limit 2^40)", name);
  if (!is_aligned(p, bytes_of(dtype))) return fail(FLCE_ERR_UNSUPPORTED, "%s must be naturally aligned", name);
  return FLCE_OK;
}

// A result in an input's place: every element has to lie where it did (a single row has no stride).
flce_status_t check_in_place(const char* name, const void* p, int dtype, int64_t ld, const char* result,
                             const void* out, int out_dtype, int64_t ldo, int64_t M) {
  if (p == out && (dtype != out_dtype || (M > 1 && ld != ldo)))
    return fail(FLCE_ERR_INVALID_VALUE, "%s in %s's place must have its type and row stride", result, name);
  return FLCE_OK;
}

// Whether 8 elements can be moved by whole 16-byte accesses.
bool vectors(const void* p, int dtype, int64_t ld) {
  return !p || (is_aligned(p, 16) && ld * int64_t(bytes_of(dtype)) % 16 == 0);
}

// An operand of the matrix product (bf16): its rows are loaded 16 bytes at a time.
flce_status_t check_operand(const char* name, const void* p, int64_t ld, int64_t cols) {
  if (!p) return fail(FLCE_ERR_INVALID_VALUE, "%s is NULL", name);
  if (ld < cols)
    return fail(FLCE_ERR_INVALID_VALUE, "%s: row stride %lld is below its %lld columns", name, (long long)ld,
                (long long)cols);
  if (ld % 8 != 0 || !is_aligned(p, 16))
    return fail(FLCE_ERR_UNSUPPORTED, "%s: rows must be 16-byte aligned", name);
  if (ld > kMaxOperandStride) return fail(FLCE_ERR_UNSUPPORTED, "%s: row stride too large (limit 2^21)", name);
  return FLCE_OK;
}

flce_status_t check_workspace(const void* p, size_t have, size_t need, const char* what) {
  if (need == 0) return FLCE_OK;
  if (!p) return fail(FLCE_ERR_INVALID_VALUE, "workspace is NULL");
  if (!is_aligned(p, kAlign)) return fail(FLCE_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
  if (have < need)
    return fail(FLCE_ERR_WORKSPACE_TOO_SMALL, "%s needs %zu workspace bytes, got %zu", what, need, have);
  return FLCE_OK;
}

// ---------------------------------------------------------------- matrix product
flce_status_t check_linear(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N <= 0 || K <= 0)
    return fail(FLCE_ERR_INVALID_VALUE, "M must be >= 0, N and K positive (got M=%lld N=%lld K=%lld)", (long long)M,
                (long long)N, (long long)K);
  if (M > flce::kMaxRows || N > flce::kMaxHidden || K > flce::kMaxHidden)
    return fail(FLCE_ERR_UNSUPPORTED, "shape too large (limits M <= 2^30, N, K <= 2^20)");
  if (K % 8 != 0) return fail(FLCE_ERR_UNSUPPORTED, "K must be a multiple of 8 (got %lld)", (long long)K);
  return FLCE_OK;
}
bool is_activation(int a) { return a >= FLCE_ACT_NONE && a <= FLCE_ACT_SILU; }

flce_status_t check_grid(const flce::LinearPlan& p, int64_t M, int64_t N) {
  if (!flce::linear_fits(p, M, N))
    return fail(FLCE_ERR_UNSUPPORTED, "too many tiles for one launch (%lld x %lld)", (long long)M, (long long)N);
  return FLCE_OK;
}

// What the backward keeps in its workspace.
struct LinearBackwardLayout {
  flce::LinearPlan dx, dw;
  int64_t ldd;
  int groups;
  size_t off_sum, off_dx, off_dw, total;
};
LinearBackwardLayout linear_backward_layout(int64_t M, int64_t N, int64_t K) {
  LinearBackwardLayout L;
  flce::linear_backward_plans(M, N, K, &L.dx, &L.dw);
  if (M > 0 && flce::linear_takes_few_dx(M, K)) L.dx = flce::linear_few_dx_plan(M, N, K);
  L.ldd = (N + 7) / 8 * 8;
  L.groups = flce::linear_slope_groups(M, N);
  L.off_sum = align_up(size_t(M) * size_t(L.ldd) * 2);
  L.off_dx = L.off_sum + align_up(size_t(L.groups) * size_t(N) * 4);
  L.off_dw = L.off_dx + align_up(flce::linear_part_bytes(L.dx, M, K));
  L.total = L.off_dw + align_up(flce::linear_part_bytes(L.dw, N, K));
  return L;
}

}  // namespace

extern "C" {

flce_status_t flce_dropout(const void* x, int x_dtype, int64_t ldx, const void* residual, int residual_dtype,
                           int64_t ldr, int64_t M, int64_t H, double p, uint64_t seed, const uint64_t* seed_at,
                           uint64_t offset, void* y, int y_dtype, int64_t ldy, hipStream_t stream) {
  if (M < 0 || H <= 0)
    return fail(FLCE_ERR_INVALID_VALUE, "rows must be >= 0 and columns positive (got %lld x %lld)", (long long)M,
                (long long)H);
  if (M > flce::kMaxRows || H > flce::kMaxHidden)
    return fail(FLCE_ERR_UNSUPPORTED, "matrix too large (limits: 2^30 rows, 2^20 columns)");
  if (!is_dtype(x_dtype) || !is_dtype(y_dtype) || (residual && !is_dtype(residual_dtype)))
    return fail(FLCE_ERR_INVALID_VALUE, "unknown element type");
  if (!(p >= 0.0 && p <= 1.0)) return fail(FLCE_ERR_INVALID_VALUE, "p must be between 0 and 1");
  if (!is_aligned(seed_at, 8)) return fail(FLCE_ERR_UNSUPPORTED, "seed_at must be 8-byte aligned");
  if (M == 0) return ok();
  flce_status_t st;
  if ((st = check_matrix("x", x, x_dtype, ldx, H)) != FLCE_OK) return st;
  if ((st = check_matrix("y", y, y_dtype, ldy, H)) != FLCE_OK) return st;
  if (residual && (st = check_matrix("residual", residual, residual_dtype, ldr, H)) != FLCE_OK) return st;
  if ((st = check_in_place("x", x, x_dtype, ldx, "y", y, y_dtype, ldy, M)) != FLCE_OK) return st;
  if ((st = check_in_place("residual", residual, residual_dtype, ldr, "y", y, y_dtype, ldy, M)) != FLCE_OK) return st;
  flce::DropoutArgs a{};
  a.x = x;
  a.ldx = long(ldx);
  a.residual = residual;
  a.ldr = long(ldr);
  a.y = y;
  a.ldy = long(ldy);
  a.M = long(M);
  a.H = int(H);
  a.threshold = uint32_t(std::nearbyint(p * 65536.0));
  a.up = a.threshold < 65536u ? float(65536.0 / (65536.0 - a.threshold)) : 0.f;
  a.seed = seed;
  a.seed_at = seed_at;
  a.offset = offset;
  const bool vec = H % 8 == 0 && vectors(x, x_dtype, ldx) && vectors(y, y_dtype, ldy) &&
                   vectors(residual, residual_dtype, ldr);
  const hipError_t e = flce::launch_dropout(a, x_dtype, residual ? residual_dtype : flce::kNoResidual, y_dtype, vec,
                                            stream);
  if (e != hipSuccess) return hip_fail(e, "dropout kernel launch");
  return ok();
}

flce_status_t flce_linear_workspace(int64_t M, int64_t N, int64_t K, size_t* fwd_bytes, size_t* bwd_bytes) {
  flce_status_t st = check_linear(M, N, K);
  if (st != FLCE_OK) return st;
  if (fwd_bytes) {
    *fwd_bytes = 0;
    if (!flce::linear_takes_few(M, N, K)) {
      const flce::LinearPlan p = flce::linear_forward_plan(M, N, K);
      if ((st = check_grid(p, M, N)) != FLCE_OK) return st;
      *fwd_bytes = align_up(flce::linear_part_bytes(p, M, N));
    }
  }
  if (bwd_bytes) {
    const LinearBackwardLayout L = linear_backward_layout(M, N, K);
    if (!flce::linear_takes_few_dx(M, K) && (st = check_grid(L.dx, M, K)) != FLCE_OK) return st;
    if ((st = check_grid(L.dw, N, K)) != FLCE_OK) return st;
    *bwd_bytes = L.total;
  }
  return ok();
}

flce_status_t flce_linear_forward(const void* X, int64_t ldx, const void* W, int64_t ldw, const void* bias,
                                  int bias_dtype, int activation, const void* residual, int residual_dtype,
                                  int64_t ldr, int64_t M, int64_t N, int64_t K, void* out, int out_dtype, int64_t ldo,
                                  void* pre, int64_t ldp, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream) {
  flce_status_t st = check_linear(M, N, K);
  if (st != FLCE_OK) return st;
  if (!is_dtype(out_dtype) || (bias && !is_dtype(bias_dtype)) || (residual && !is_dtype(residual_dtype)))
    return fail(FLCE_ERR_INVALID_VALUE, "unknown element type");
  if (!is_activation(activation)) return fail(FLCE_ERR_INVALID_VALUE, "unknown activation %d", activation);
  if (M == 0) return ok();
  if ((st = check_operand("X", X, ldx, K)) != FLCE_OK) return st;
  if ((st = check_operand("W", W, ldw, K)) != FLCE_OK) return st;
  if ((st = check_matrix("out", out, out_dtype, ldo, N)) != FLCE_OK) return st;
  if (residual && (st = check_matrix("residual", residual, residual_dtype, ldr, N)) != FLCE_OK) return st;
  if ((st = check_in_place("residual", residual, residual_dtype, ldr, "out", out, out_dtype, ldo, M)) != FLCE_OK)
    return st;
  if (pre && (st = check_matrix("pre", pre, FLCE_BF16, ldp, N)) != FLCE_OK) return st;
  if (!is_aligned(bias, bias ? bytes_of(bias_dtype) : 1))
    return fail(FLCE_ERR_UNSUPPORTED, "bias must be naturally aligned");
  const flce::LinearProduct a{static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(W), long(ldx), long(ldw),
                              int(M), int(N), int(K), int(K), int(K)};
  flce::LinearEpilogue e{};
  e.bias = bias;
  e.bias_dtype = bias_dtype;
  e.act = activation;
  e.residual = residual;
  e.residual_dtype = residual_dtype;
  e.ldr = long(ldr);
  e.out = out;
  e.out_dtype = out_dtype;
  e.ldo = long(ldo);
  e.pre = static_cast<uint16_t*>(pre);
  e.ldp = long(ldp);
  hipError_t err;
  if (flce::linear_takes_few(M, N, K)) {
    err = flce::launch_linear_few(a, e, stream);
  } else {
    const flce::LinearPlan plan = flce::linear_forward_plan(M, N, K);
    if ((st = check_grid(plan, M, N)) != FLCE_OK) return st;
    const size_t need = flce::linear_part_bytes(plan, M, N);
    if ((st = check_workspace(workspace, workspace_bytes, need, "linear forward")) != FLCE_OK) return st;
    err = flce::launch_linear_product(a, plan, e, static_cast<float*>(workspace), stream);
  }
  if (err != hipSuccess) return hip_fail(err, "linear kernel launch");
  return ok();
}

flce_status_t flce_linear_backward(const void* dy, int dy_dtype, int64_t lddy, const void* pre, int64_t ldp,
                                   int activation, const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t M,
                                   int64_t N, int64_t K, void* dX, int64_t lddx, void* dW, int64_t lddw, void* dbias,
                                   int bias_dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  flce_status_t st = check_linear(M, N, K);
  if (st != FLCE_OK) return st;
  if (!is_dtype(dy_dtype) || (dbias && !is_dtype(bias_dtype)))
    return fail(FLCE_ERR_INVALID_VALUE, "unknown element type");
  if (!is_activation(activation)) return fail(FLCE_ERR_INVALID_VALUE, "unknown activation %d", activation);
  if (dbias && !is_aligned(dbias, bytes_of(bias_dtype)))
    return fail(FLCE_ERR_UNSUPPORTED, "dbias must be naturally aligned");
  const bool act = activation != FLCE_ACT_NONE;
  if (M > 0) {
    if ((st = check_matrix("dy", dy, dy_dtype, lddy, N)) != FLCE_OK) return st;
    if (act && (st = check_matrix("pre", pre, FLCE_BF16, ldp, N)) != FLCE_OK) return st;
    if (dW && (st = check_operand("X", X, ldx, K)) != FLCE_OK) return st;
    if (dX && (st = check_operand("W", W, ldw, K)) != FLCE_OK) return st;
    if (dX && (st = check_matrix("dX", dX, FLCE_BF16, lddx, K)) != FLCE_OK) return st;
  }
  if (dW && (st = check_matrix("dW", dW, FLCE_BF16, lddw, K)) != FLCE_OK) return st;
  const LinearBackwardLayout L = linear_backward_layout(M, N, K);
  if (dX && !flce::linear_takes_few_dx(M, K) && (st = check_grid(L.dx, M, K)) != FLCE_OK) return st;
  if (dW && (st = check_grid(L.dw, N, K)) != FLCE_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, L.total, "linear backward")) != FLCE_OK) return st;
  char* ws = static_cast<char*>(workspace);

  // dy itself where it already is what the products read
  const bool as_is = !act && dy_dtype == FLCE_BF16 && N % 8 == 0 && lddy % 8 == 0 && is_aligned(dy, 16) &&
                     lddy <= kMaxOperandStride;
  const uint16_t* dpre = as_is ? static_cast<const uint16_t*>(dy) : reinterpret_cast<const uint16_t*>(ws);
  const int64_t ldd = as_is ? lddy : L.ldd;
  const bool few = flce::linear_takes_few_dx(M, K);
  const bool write = !as_is && (dW || (dX && !few));
  if (M > 0 && (write || dbias)) {
    flce::LinearSlopeArgs a{};
    a.dy = dy;
    a.dy_dtype = dy_dtype;
    a.lddy = long(lddy);
    a.pre = act ? static_cast<const uint16_t*>(pre) : nullptr;
    a.ldp = long(ldp);
    a.act = activation;
    a.M = long(M);
    a.N = int(N);
    a.dpre = write ? reinterpret_cast<uint16_t*>(ws) : nullptr;
    a.ldd = long(L.ldd);
    a.part = dbias ? reinterpret_cast<float*>(ws + L.off_sum) : nullptr;
    a.groups = L.groups;
    a.vec = N % 8 == 0 && vectors(dy, dy_dtype, lddy) && vectors(a.pre, FLCE_BF16, ldp);
    const hipError_t e = flce::launch_linear_slope(a, stream);
    if (e != hipSuccess) return hip_fail(e, "activation gradient kernel launch");
  }
  if (dX && M > 0 && few) {
    flce::LinearFewDx a{};
    a.dy = dy;
    a.dy_dtype = dy_dtype;
    a.lddy = long(lddy);
    a.pre = act ? static_cast<const uint16_t*>(pre) : nullptr;
    a.ldp = long(ldp);
    a.act = activation;
    a.w = static_cast<const uint16_t*>(W);
    a.ldw = long(ldw);
    a.M = int(M);
    a.N = int(N);
    a.K = int(K);
    a.dx = static_cast<uint16_t*>(dX);
    a.lddx = long(lddx);
    a.part = reinterpret_cast<float*>(ws + L.off_dx);
    const hipError_t e = flce::launch_linear_few_dx(a, L.dx, stream);
    if (e != hipSuccess) return hip_fail(e, "linear gradient kernel launch");
  }
  flce::LinearGradArgs g{};
  const int64_t N8 = (N + 7) / 8 * 8;
  if (dX && M > 0 && !few) {
    g.dx = {dpre, static_cast<const uint16_t*>(W), long(ldd), long(ldw), int(M), int(K), int(N8), int(N8), int(N)};
    g.out_dx.out = dX;
    g.out_dx.out_dtype = FLCE_BF16;
    g.out_dx.ldo = long(lddx);
    g.n_dx = int(flce::linear_workgroups(L.dx, M, K));
  }
  if (dW) {
    g.dw = {dpre, static_cast<const uint16_t*>(X), long(ldd), long(ldx), int(N), int(K), int(M), int(M), int(M)};
    g.out_dw.out = dW;
    g.out_dw.out_dtype = FLCE_BF16;
    g.out_dw.ldo = long(lddw);
    g.n_dw = int(flce::linear_workgroups(L.dw, N, K));
  }
  g.plan_dx = L.dx;
  g.plan_dw = L.dw;
  g.part_dx = reinterpret_cast<float*>(ws + L.off_dx);
  g.part_dw = reinterpret_cast<float*>(ws + L.off_dw);
  g.bias = {reinterpret_cast<const float*>(ws + L.off_sum), M > 0 ? L.groups : 0, int(N), dbias, bias_dtype};
  const hipError_t e = flce::launch_linear_grad(g, stream);
  if (e != hipSuccess) return hip_fail(e, "linear gradient kernel launch");
  return ok();
}

}  // extern "C"

namespace {

// ---------------------------------------------------------------- log-probs from logits
flce_status_t check_logits(int64_t M, int64_t V, int64_t n_tokens, int64_t n_top, float scale) {
  if (M < 0 || V <= 0)
    return fail(FLCE_ERR_INVALID_VALUE, "M must be >= 0 and V positive (got M=%lld V=%lld)", (long long)M,
                (long long)V);
  if (M > flce::kMaxRows || V > flce::kMaxVocab)
    return fail(FLCE_ERR_UNSUPPORTED, "shape too large (limits M, V <= 2^30)");
  if (n_tokens < 0 || n_top < 0)
    return fail(FLCE_ERR_INVALID_VALUE, "n_tokens and n_top must be >= 0");
  if (n_tokens > flce::kMaxTokens || n_top > flce::kMaxTop)
    return fail(FLCE_ERR_UNSUPPORTED, "at most %d tokens and %d alternatives a row", flce::kMaxTokens, flce::kMaxTop);
  if (n_top > V)
    return fail(FLCE_ERR_INVALID_VALUE, "n_top %lld exceeds the %lld logits of a row", (long long)n_top, (long long)V);
  if (!(scale > 0.f && scale <= 1.8446744e19f))
    return fail(FLCE_ERR_INVALID_VALUE, "scale must be positive and at most 2^64");
  return FLCE_OK;
}

struct LogprobLayout {
  int parts, part_len;
  size_t off_top, total;
};
LogprobLayout logprob_layout(int64_t M, int64_t V, int64_t n_top) {
  LogprobLayout L;
  flce::token_logprob_split(M, V, int(n_top), &L.parts, &L.part_len);
  const size_t items = L.parts > 1 ? size_t(M) * size_t(L.parts) : 0;
  L.off_top = align_up(items * 3 * 4);
  L.total = L.off_top + align_up(items * size_t(n_top) * 8);
  return L;
}

}  // namespace

extern "C" {

flce_status_t flce_token_logprobs_workspace(int64_t M, int64_t V, int64_t n_top, size_t* bytes) {
  flce_status_t st = check_logits(M, V, 0, n_top, 1.f);
  if (st != FLCE_OK) return st;
  if (!bytes) return fail(FLCE_ERR_INVALID_VALUE, "bytes is NULL");
  *bytes = logprob_layout(M, V, n_top).total;
  return ok();
}

flce_status_t flce_token_logprobs(const void* logits, int dtype, int64_t ldl, int64_t M, int64_t V,
                                  const int64_t* tokens, int64_t n_tokens, int64_t ignore_index, float scale,
                                  int64_t n_top, float* logprob, float* lse, float* entropy, float* stats,
                                  int64_t* top_ids, float* top_logprob, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream) {
  flce_status_t st = check_logits(M, V, n_tokens, n_top, scale);
  if (st != FLCE_OK) return st;
  if (!is_dtype(dtype)) return fail(FLCE_ERR_INVALID_VALUE, "unknown element type");
  if (M == 0) return ok();
  if ((st = check_matrix("logits", logits, dtype, ldl, V)) != FLCE_OK) return st;
  if (!lse || !stats || (n_tokens && (!tokens || !logprob)) || (n_top && (!top_ids || !top_logprob)))
    return fail(FLCE_ERR_INVALID_VALUE, "NULL pointer among tokens, logprob, lse, stats, top_ids, top_logprob");
  if (!is_aligned(tokens, 8) || !is_aligned(top_ids, 8) || !is_aligned(logprob, 4) || !is_aligned(lse, 4) ||
      !is_aligned(entropy, 4) || !is_aligned(stats, 4) || !is_aligned(top_logprob, 4))
    return fail(FLCE_ERR_UNSUPPORTED, "tokens and outputs must be naturally aligned");
  const LogprobLayout L = logprob_layout(M, V, n_top);
  if ((st = check_workspace(workspace, workspace_bytes, L.total, "token log-probs")) != FLCE_OK) return st;
  flce::TokenLogprobArgs a{};
  a.logits = logits;
  a.ldl = long(ldl);
  a.M = long(M);
  a.V = int(V);
  a.tokens = tokens;
  a.n_tokens = int(n_tokens);
  a.ignore_index = ignore_index;
  a.scale = scale;
  a.n_top = int(n_top);
  a.logprob = logprob;
  a.lse = lse;
  a.entropy = entropy;
  a.stats = stats;
  a.top_ids = top_ids;
  a.top_logprob = top_logprob;
  a.parts = L.parts;
  a.part_len = L.part_len;
  a.part_sums = static_cast<float*>(workspace);
  a.part_top = reinterpret_cast<unsigned long long*>(static_cast<char*>(workspace) + L.off_top);
  const hipError_t e = flce::launch_token_logprobs(a, dtype, stream);
  if (e != hipSuccess) return hip_fail(e, "token log-prob kernel launch");
  return ok();
}

flce_status_t flce_token_logprobs_backward(const void* logits, int dtype, int64_t ldl, int64_t M, int64_t V,
                                           const int64_t* tokens, int64_t n_tokens, int64_t ignore_index, float scale,
                                           const float* stats, const float* entropy, const int64_t* top_ids,
                                           int64_t n_top, const float* grad_logprob, const float* grad_top,
                                           const float* grad_entropy, const float* grad_lse, void* dlogits,
                                           int64_t ldd, hipStream_t stream) {
  flce_status_t st = check_logits(M, V, n_tokens, n_top, scale);
  if (st != FLCE_OK) return st;
  if (!is_dtype(dtype)) return fail(FLCE_ERR_INVALID_VALUE, "unknown element type");
  if (M == 0) return ok();
  if ((st = check_matrix("logits", logits, dtype, ldl, V)) != FLCE_OK) return st;
  if ((st = check_matrix("dlogits", dlogits, dtype, ldd, V)) != FLCE_OK) return st;
  if ((st = check_in_place("logits", logits, dtype, ldl, "dlogits", dlogits, dtype, ldd, M)) != FLCE_OK) return st;
  if (!stats) return fail(FLCE_ERR_INVALID_VALUE, "stats is NULL");
  if ((n_tokens && !tokens) || (grad_entropy && !entropy) || (grad_top && n_top && !top_ids))
    return fail(FLCE_ERR_INVALID_VALUE, "NULL pointer among tokens, entropy, top_ids");
  if (!is_aligned(tokens, 8) || !is_aligned(top_ids, 8) || !is_aligned(stats, 4) || !is_aligned(entropy, 4) ||
      !is_aligned(grad_logprob, 4) || !is_aligned(grad_top, 4) || !is_aligned(grad_entropy, 4) ||
      !is_aligned(grad_lse, 4))
    return fail(FLCE_ERR_UNSUPPORTED, "tokens, statistics and gradients must be naturally aligned");
  flce::TokenLogprobGradArgs a{};
  a.logits = logits;
  a.ldl = long(ldl);
  a.M = long(M);
  a.V = int(V);
  a.tokens = tokens;
  a.n_tokens = grad_logprob ? int(n_tokens) : 0;
  a.ignore_index = ignore_index;
  a.scale = scale;
  a.stats = stats;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.n_top = grad_top ? int(n_top) : 0;
  a.grad_logprob = grad_logprob;
  a.grad_top = grad_top;
  a.grad_entropy = grad_entropy;
  a.grad_lse = grad_lse;
  a.dlogits = dlogits;
  a.ldd = long(ldd);
  const hipError_t e = flce::launch_token_logprobs_grad(a, dtype, stream);
  if (e != hipSuccess) return hip_fail(e, "token log-prob gradient kernel launch");
  return ok();
}

}  // extern "C"
