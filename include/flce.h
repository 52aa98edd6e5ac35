/*
 * libflce: fused LM-head linear + cross-entropy (per-token log-prob, log-sum-exp
 * and optional entropy) for AMD gfx950, forward and backward, without ever
 * materialising the [M, V] logits.
 *
 * The operation (Liger-Kernel commit "native Blackwell tensor-parallel fused
 * scaled linear cross-entropy", section "Summary": the classifier GEMM fused with
 * NLL/LSE and optional entropy; SkyRL PR 2141 "perf(megatron): autotune fused
 * LM-head Triton kernels", sections "Summary"/"Overview": per-token log-probs,
 * optional entropy via compute_entropy, LSE seeded from the true row maximum):
 *
 *   z[m, v]    = scale * sum_k X[m, k] * W[v, k]        bf16 inputs, fp32 accumulation
 *   lse[m]     = log sum_v exp z[m, v]
 *   logprob[m] = z[m, t[m]] - lse[m]
 *   entropy[m] = -sum_v p[m, v] log p[m, v],  p = softmax(z[m, :])
 *
 * A row m is valid iff t[m] != ignore_index and 0 <= t[m] < V.  Invalid rows get
 * logprob = 0 and entropy = 0 (lse is still written) and contribute nothing to
 * the gradients.
 *
 * M = 0 (an empty batch) is accepted everywhere: workspace sizes are 0, the forward
 * calls return FLCE_OK without touching any pointer, and the backward writes dW = 0
 * (the only output with elements).  H and V must be positive.
 *
 * Backward, for a loss L with dL/dlogprob = grad_logprob and dL/dentropy =
 * grad_entropy (Liger-Kernel PR 1294 "Triton MoE improvements and chunked GRPO
 * improvements", "Kernel design notes": logits tiles are recomputed to form
 * grad_logits in the input dtype, then the two grad GEMMs):
 *
 *   dz[m, v] = a[m] (1[v = t[m]] - p[m, v]) + b[m] p[m, v] (E[m] - z[m, v])
 *   a = grad_logprob * valid, b = grad_entropy * valid, E = lse - entropy
 *   dX = scale * dz W,  dW = scale * dz^T X            (bf16 results)
 *
 * Layouts: every matrix is row-major and contiguous.  X is [M, H] bf16, W is
 * [V, H] bf16 (the nn.Linear weight layout, logits = X W^T), targets is [M]
 * int64.  All pointers are device pointers except the size_t outputs of
 * flce_workspace_query.
 *
 * Ownership and ordering: the caller owns every buffer (inputs, outputs and the
 * workspace).  The library never allocates or frees device memory and never
 * synchronises: a call validates its arguments on the host, enqueues kernels on
 * `stream` and returns; results are valid in stream order.  Inputs are never
 * written.  Outputs are overwritten, not accumulated.  Workspace contents are not
 * preserved between calls; forward -> backward state travels only through the
 * caller-held lse and entropy outputs.  Calls on different streams may run
 * concurrently if they use different workspaces and outputs.
 *
 * Errors: return codes only; nothing aborts.  All argument checks happen on the
 * host before any HIP call, so a rejected call enqueues nothing.  After
 * FLCE_ERR_HIP some kernels of the call may already have been enqueued.
 * flce_last_error_message() gives a thread-local description of the last failure.
 */
#ifndef LIBFLCE_FLCE_H
#define LIBFLCE_FLCE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct ihipStream_t; /* hipStream_t is `struct ihipStream_t *`; NULL = default stream */

typedef enum {
  FLCE_OK = 0,
  FLCE_ERR_INVALID_VALUE = 1,       /* NULL pointer, size <= 0, bad flag, non-finite scale */
  FLCE_ERR_UNSUPPORTED = 2,         /* H % 8 != 0, pointer not 16-byte aligned, size too large */
  FLCE_ERR_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes below what the call needs */
  FLCE_ERR_HIP = 4                  /* a HIP launch failed; see flce_last_error_message() */
} flce_status_t;

/*
 * Workspace bytes needed by flce_forward (*fwd_bytes) and the preferred size for
 * flce_backward (*bwd_bytes) for this problem shape.  One buffer of
 * max(*fwd_bytes, *bwd_bytes) serves both.  Either output pointer may be NULL.
 * Sizes accepted by every call: 0 <= M <= 2^30 (M = 0 is an empty batch),
 * 8 <= H <= 2^20 with H % 8 == 0, 1 <= V <= 2^30.  Negative M, or H or V <= 0:
 * FLCE_ERR_INVALID_VALUE; larger sizes, or H not a multiple of 8:
 * FLCE_ERR_UNSUPPORTED.  A dispatch covers at most 2^32 - 1 work-items, so very
 * large problems run in more token waves (and narrower chunks) than the workspace
 * alone would need; *fwd_bytes is the size of the tallest such forward wave.  The
 * one-launch calls (flce_forward_partials and its shard form, flce_forward_merge)
 * return FLCE_ERR_UNSUPPORTED for a batch taller than one launch can take.
 */
flce_status_t flce_workspace_query(int64_t M, int64_t H, int64_t V, int compute_entropy,
                                   size_t* fwd_bytes, size_t* bwd_bytes);

/*
 * Backward workspace.  The backward runs in token waves and vocabulary chunks whose
 * sizes it derives from the workspace it is given (the token-wave scheduling of the
 * Liger-Kernel commit "native Blackwell tensor-parallel fused scaled linear
 * cross-entropy", sections "Summary", "Implementation / Backward" and "Correctness":
 * dW stored by the first wave and added to by later ones; Liger-Kernel PR 1294,
 * "Kernel design notes": d-logits in the input dtype in a reusable buffer).  The
 * workspace holds the bf16 d-logits of one wave over one chunk; an fp32 dX
 * accumulator for one wave's rows when a wave takes more than one chunk; when
 * there is more than one wave, an fp32 dW accumulator of V x H; and 256 bytes of
 * counters with which the d-logit and dW kernels hand out their last tiles.  The preferred size
 * (*bwd_bytes of flce_workspace_query) is one wave of every row with up to 4 GiB of
 * d-logits per chunk (every column at once when they fit).  With less, the call
 * takes the schedule that fits and moves the fewest extra bytes: narrower chunks, or
 * waves of 256 to 16384 rows.  Schedules whose steps (one wave over one chunk) are at
 * most 8e12 FLOP (6 x rows x H x chunk) may also run pipelined when two d-logit
 * buffers fit: one launch per step computes the step's dW and dX together with the
 * next step's d-logits; the same fewest-extra-bytes rule, which counts launches,
 * picks between the kinds.  The minimum is the smallest of: one wave with 256-column
 * chunks (d-logits + fp32 dX accumulator of M rows), one wave with every column
 * (d-logits only), 256-row waves with 256-column chunks or with every column (+ the
 * fp32 dW accumulator): once M > 256 it is at most 4 V H + 1024 H + 131328 bytes (each
 * part rounded up to 256 bytes), whatever M.  Results of different schedules differ
 * only by fp32 summation order (dX across chunks, dW across waves); every schedule is
 * deterministic, and a pipelined schedule gives the same bits as three launches per
 * step with the same waves and chunks.
 */
flce_status_t flce_backward_workspace_min(int64_t M, int64_t H, int64_t V, size_t* bytes);

/* Chunk width (vocabulary columns) flce_backward would use with this workspace;
 * FLCE_ERR_WORKSPACE_TOO_SMALL below the minimum. */
flce_status_t flce_backward_chunk_cols(int64_t M, int64_t H, int64_t V, size_t workspace_bytes,
                                       int64_t* chunk_cols);

/* The whole schedule flce_backward would run with this workspace: token rows per wave,
 * chunk width, and whether it runs pipelined (1: one launch per step, the dW and dX
 * tiles of one step with the d-logit tiles of the next, over two d-logit buffers) or
 * as three launches per step (0).  Any output may be NULL; FLCE_ERR_WORKSPACE_TOO_SMALL
 * below the minimum. */
flce_status_t flce_backward_schedule(int64_t M, int64_t H, int64_t V, size_t workspace_bytes,
                                     int64_t* rows, int64_t* chunk_cols, int* pipelined);

/* Token rows per wave flce_backward would use with this workspace (a multiple of 256;
 * M rounded up to 256 means one wave); FLCE_ERR_WORKSPACE_TOO_SMALL below the minimum. */
flce_status_t flce_backward_wave_rows(int64_t M, int64_t H, int64_t V, size_t workspace_bytes,
                                      int64_t* rows);

/*
 * Smallest workspace flce_forward accepts, and the wave height it uses with a given
 * workspace.  The forward walks the tokens in waves (the token-wave scheduling of
 * the Liger-Kernel commit "native Blackwell tensor-parallel fused scaled linear
 * cross-entropy", sections "Summary" and "Correctness": 4K waves, two-wave tails):
 * a wave is a multiple of 256 rows whose per-tile partials (12 bytes per row per
 * 256 vocabulary columns with entropy, 8 without), target logits (4 bytes per row)
 * and 256 bytes of tile-queue counters fit in the workspace.  The size
 * from flce_workspace_query takes all rows in one wave; the minimum takes 256.
 * Results are bitwise identical for every wave height: a row's tiles and merge do
 * not depend on the wave it falls in.
 */
flce_status_t flce_forward_workspace_min(int64_t M, int64_t H, int64_t V, int compute_entropy,
                                         size_t* bytes);

/* Rows per token wave flce_forward would use with this workspace (a multiple of 256,
 * at most M rounded up to 256); FLCE_ERR_WORKSPACE_TOO_SMALL below the minimum. */
flce_status_t flce_forward_wave_rows(int64_t M, int64_t H, int64_t V, int compute_entropy,
                                     size_t workspace_bytes, int64_t* rows);

/*
 * Forward.  Writes logprob[M], lse[M] and, if compute_entropy == 1, entropy[M]
 * (all fp32).  entropy may be NULL only when compute_entropy == 0.
 * scale is the temperature factor applied to the fp32 accumulator (1/T).
 * workspace: device memory of at least flce_forward_workspace_min bytes (the
 * *fwd_bytes of flce_workspace_query runs every row in one wave), 256-byte aligned.
 */
flce_status_t flce_forward(const void* X, const void* W, const int64_t* targets,
                           int64_t M, int64_t H, int64_t V, int64_t ignore_index, float scale,
                           int compute_entropy, float* logprob, float* lse, float* entropy,
                           void* workspace, size_t workspace_bytes, struct ihipStream_t* stream);

/*
 * flce_forward for callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  It takes no
 * workspace: the partials go to a static device scratch array of the library, 32 MiB
 * (FLCE_NOALLOC_SCRATCH_BYTES) on each GPU it runs on, held until the process ends,
 * and the token waves are sized to it.  The call allocates and frees nothing; it
 * uses the scratch of the current device, so `stream` must belong to that device.
 * Results are bitwise identical to flce_forward's.  Every value of the scratch a call
 * reads is written earlier in that call, so nothing needs clearing, but the scratch
 * is shared: calls that overlap on one GPU (different streams, or threads) race and
 * must be serialised by the caller.  A vocabulary whose partials of one 256-row wave
 * (12 bytes per 256 columns with entropy, 8 without, per row) exceed the scratch,
 * V above about 2.8M with entropy, is rejected with FLCE_ERR_UNSUPPORTED.  The first
 * call on a device looks the scratch's address up (hipGetSymbolAddress); a failure
 * there is FLCE_ERR_HIP.  Other arguments and errors as flce_forward.
 */
#define FLCE_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
flce_status_t flce_forward_noalloc(const void* X, const void* W, const int64_t* targets,
                                   int64_t M, int64_t H, int64_t V, int64_t ignore_index,
                                   float scale, int compute_entropy, float* logprob, float* lse,
                                   float* entropy, struct ihipStream_t* stream);

/*
 * The two halves of flce_forward, for callers that exchange or inspect the
 * per-tile statistics (a vocabulary-sharded caller gathers them across shards
 * before merging).  flce_forward_partials runs the fused GEMM + online-softmax
 * kernel over all rows in one wave (the workspace must hold *fwd_bytes of
 * flce_workspace_query) and leaves in the workspace, for every row m and
 * 256-column vocabulary tile j (j < ceil(V / 256), Mpad = 256 * ceil(M / 256)),
 * at float offsets
 *   j * Mpad + m                       max_v z[m, v] over the tile
 *   (n_vt + j) * Mpad + m              sum_v exp(z[m, v] - max)
 *   (2 n_vt + j) * Mpad + m            sum_v exp(z[m, v] - max) (z[m, v] - max)  (entropy only)
 * and after the 2 (or 3) partial arrays (each rounded up to 256 bytes) the
 * target logit z[m, t[m]] of every valid row (Mpad floats, rounded up to 256 bytes),
 * then the 256 bytes of counters with which the tile kernel hands out its last tiles.  flce_forward_merge turns them into
 * logprob, lse and entropy; its arguments must match the partials call.
 */
flce_status_t flce_forward_partials(const void* X, const void* W, const int64_t* targets,
                                    int64_t M, int64_t H, int64_t V, int64_t ignore_index,
                                    float scale, int compute_entropy, void* workspace,
                                    size_t workspace_bytes, struct ihipStream_t* stream);

flce_status_t flce_forward_merge(const int64_t* targets, int64_t M, int64_t H, int64_t V,
                                 int64_t ignore_index, int compute_entropy, float* logprob,
                                 float* lse, float* entropy, const void* workspace,
                                 size_t workspace_bytes, struct ihipStream_t* stream);

/*
 * Backward.  Recomputes the logits, forms dz and writes dX [M, H] and dW [V, H]
 * in bf16.  lse comes from flce_forward; entropy (from flce_forward with
 * compute_entropy == 1) is required iff grad_entropy != NULL.  grad_logprob and
 * grad_entropy are fp32 [M]; NULL means zero (both NULL writes zero gradients).
 * workspace: at least flce_backward_workspace_min bytes, 256-byte aligned.
 */
flce_status_t flce_backward(const void* X, const void* W, const int64_t* targets,
                            int64_t M, int64_t H, int64_t V, int64_t ignore_index, float scale,
                            const float* lse, const float* entropy,
                            const float* grad_logprob, const float* grad_entropy,
                            void* dX, void* dW,
                            void* workspace, size_t workspace_bytes, struct ihipStream_t* stream);

/*
 * Vocabulary shards (the tensor-parallel split of Liger-Kernel "native Blackwell
 * tensor-parallel fused scaled linear cross-entropy", sections "Summary" and
 * "Implementation": each rank holds a contiguous block of W's rows; SkyRL PR 2141,
 * review of the TP-aware adapter: the rank only shifts vocabulary ids).  A shard is
 * W rows [v_offset, v_offset + V_shard) of a vocabulary of V_total ids; targets stay
 * global ids.  The three calls below are what one rank runs; the exchange between
 * ranks (an all-gather of the partials, a sum of the dX partials) belongs to the
 * caller's communication library.
 *
 * flce_forward_partials_shard: as flce_forward_partials for W_shard [V_shard, H]
 * (the workspace layout is that of flce_forward_partials with V = V_shard; its
 * size is *fwd_bytes of flce_workspace_query(M, H, V_shard, ...)).  The target
 * logit of row m is written only if this shard owns t[m].  v_offset must be in
 * [0, 2^30 - V_shard].
 */
flce_status_t flce_forward_partials_shard(const void* X, const void* W_shard,
                                          const int64_t* targets, int64_t M, int64_t H,
                                          int64_t V_shard, int64_t v_offset,
                                          int64_t ignore_index, float scale, int compute_entropy,
                                          void* workspace, size_t workspace_bytes,
                                          struct ihipStream_t* stream);

/*
 * Merge of the gathered partials of n_shards shards (1 <= n_shards <= 64) into
 * logprob, lse and entropy over the whole vocabulary.  shard_offsets is a HOST
 * array of n_shards + 1 ids: shard r covers [shard_offsets[r], shard_offsets[r + 1]),
 * shard_offsets[0] = 0 and the sequence strictly increases (V_total =
 * shard_offsets[n_shards]).  Shard r's partials, exactly as
 * flce_forward_partials_shard left them, start at byte r * shard_stride_bytes of
 * `gathered` (device memory of n_shards * shard_stride_bytes bytes, 256-byte
 * aligned; the stride is a multiple of 256 and at least every shard's forward
 * workspace size).  Validity uses V_total; the target logit comes from the owning
 * shard.  Results match flce_forward on the whole vocabulary up to fp32 summation
 * order.
 */
flce_status_t flce_forward_merge_shards(const int64_t* targets, int64_t M, int64_t n_shards,
                                        const int64_t* shard_offsets, int64_t ignore_index,
                                        int compute_entropy, float* logprob, float* lse,
                                        float* entropy, const void* gathered,
                                        size_t shard_stride_bytes, struct ihipStream_t* stream);

/* Workspace bytes for flce_backward_shard: the minimum and the preferred size, as
 * for flce_backward but without a dX accumulator (dX_partial is the caller's fp32
 * buffer): d-logits of one wave over one chunk, plus the fp32 dW_shard accumulator
 * when the rows run in more than one wave.  Either output may be NULL. */
flce_status_t flce_backward_shard_workspace_query(int64_t M, int64_t H, int64_t V_shard,
                                                  size_t* min_bytes, size_t* preferred_bytes);

/*
 * Backward of one shard, given the global lse (and entropy) from the merge:
 * writes dW_shard [V_shard, H] bf16 (the shard's rows of dW) and this shard's
 * term of dX, dz_shard W_shard * scale, in fp32 to dX_partial [M, H]: overwritten
 * if accumulate == 0, added to if accumulate == 1 (one GPU can sum several shards
 * in a fixed order this way; across ranks the terms are summed by an all-reduce).
 * dX = sum over shards of dX_partial.  A row is valid iff t[m] != ignore_index and
 * 0 <= t[m] < V_total.  workspace: at least the minimum of
 * flce_backward_shard_workspace_query, 256-byte aligned.
 */
flce_status_t flce_backward_shard(const void* X, const void* W_shard, const int64_t* targets,
                                  int64_t M, int64_t H, int64_t V_shard, int64_t v_offset,
                                  int64_t V_total, int64_t ignore_index, float scale,
                                  const float* lse, const float* entropy,
                                  const float* grad_logprob, const float* grad_entropy,
                                  float* dX_partial, int accumulate, void* dW_shard,
                                  void* workspace, size_t workspace_bytes,
                                  struct ihipStream_t* stream);

/*
 * Scalar cross-entropy reductions over the valid rows of a forward's logprob
 * (the token-level NLL of Liger-Kernel "native Blackwell tensor-parallel fused
 * scaled linear cross-entropy", section "Summary", reduced outside the per-token
 * kernels as SkyRL PR 2141, section "Summary", keeps it).  Writes three fp64
 * values to the device array out: the sum of -logprob[m] over valid rows, the
 * number of valid rows, and their mean (NaN when no row is valid).  One
 * workgroup with a fixed summation order: the result is bitwise repeatable.
 * Validity as in flce_forward (t != ignore_index and 0 <= t < V).
 */
flce_status_t flce_nll_reduce(const float* logprob, const int64_t* targets, int64_t M,
                              int64_t V, int64_t ignore_index, double* out,
                              struct ihipStream_t* stream);

/*
 * dL/dlogprob for L = the mean NLL: grad_logprob[m] = -1/n on valid rows and 0
 * elsewhere, n read on the device from reduced[1] (the out array of
 * flce_nll_reduce), so no host synchronisation is needed; all zeros when n = 0.
 * The result is the grad_logprob argument of flce_backward.
 */
flce_status_t flce_nll_mean_grad(const int64_t* targets, int64_t M, int64_t V,
                                 int64_t ignore_index, const double* reduced,
                                 float* grad_logprob, struct ihipStream_t* stream);

/*
 * Clipped policy-gradient loss on a forward's per-token log-probs, aggregated as a
 * token mean (Liger-Kernel PR 1294, section "Chunked Triton GRPO loss": the loss on
 * top of the fused linear log-probs, settings "Setup" (loss type dapo, clip range
 * eps 0.2/0.2, num_items_in_batch) and per-token outputs "Correctness"; the page
 * gives no formulas, this is the plain clipped-surrogate reading).  Per token m,
 * valid as in flce_forward, in fp64:
 *   r = exp(logprob[m] - old_logprob[m])          (old_logprob NULL: r = 1)
 *   c = min(max(r, 1 - eps_low), 1 + eps_high)
 *   per_token_loss[m] = -min(r A[m], c A[m])      (0 on invalid rows, as fp32)
 *   is_clipped[m]     = c A[m] < r A[m]           (optional output, NULL to skip)
 * where a NaN among a valid row's inputs makes its loss (and its gradient below) NaN,
 * and four fp64 values to the device array out: the sum of the per-token loss over
 * valid rows, the number of valid rows, the number of clipped rows, and the loss
 * sum / N with N = denominator if > 0 (the caller's normaliser, e.g. the number of
 * items in the batch), else the number of valid rows; NaN when N is 0.  One
 * workgroup with a fixed summation order: bitwise repeatable.  eps_low and
 * eps_high must be finite and >= 0, denominator finite; all arrays on the device.
 */
flce_status_t flce_policy_loss_reduce(const float* logprob, const float* old_logprob,
                                      const float* advantages, const int64_t* targets,
                                      int64_t M, int64_t V, int64_t ignore_index,
                                      double eps_low, double eps_high, double denominator,
                                      float* per_token_loss, uint8_t* is_clipped, double* out,
                                      struct ihipStream_t* stream);

/*
 * dL/dlogprob of the loss of flce_policy_loss_reduce (same inputs):
 * grad_logprob[m] = -r A[m] / N on valid rows whose minimum takes the unclipped
 * term, 0 on clipped and invalid rows, all zeros when N is 0.  With denominator <= 0,
 * N is read on the device from reduced[1] (the out array of
 * flce_policy_loss_reduce), so no host synchronisation is needed; reduced may be
 * NULL when denominator > 0.  The result is the grad_logprob argument of
 * flce_backward.
 */
flce_status_t flce_policy_loss_grad(const float* logprob, const float* old_logprob,
                                    const float* advantages, const int64_t* targets, int64_t M,
                                    int64_t V, int64_t ignore_index, double eps_low,
                                    double eps_high, double denominator, const double* reduced,
                                    float* grad_logprob, struct ihipStream_t* stream);

/*
 * Element types and microscaled formats of the calls below.  A microscaled matrix keeps
 * blocks of 32 consecutive elements of a row with one power-of-two scale: the smallest 2^e
 * (-127 <= e <= 127) at which no element of the block exceeds the element format's largest
 * value (at e = 127 elements are clamped to it); elements are rounded to nearest, ties to
 * even.  Element formats: MXFP4 e2m1 (largest 6; two codes a byte, the even element in the
 * low half), MXFP8 e4m3 (largest 448), MXINT8 an integer in [-127, 127] over 64.  A block
 * that holds an infinity or a NaN stands for NaNs throughout.  Layout, row-major: codes,
 * each row padded with zeros to a whole block, and scale bytes (e + 127; 255 for NaN), each
 * row padded with zeros to a multiple of 16 bytes; flce_mx_sizes gives the bytes of a row.
 * The products below rely on the padding: a matrix quantised elsewhere must have it too.
 */
typedef enum { FLCE_BF16 = 0, FLCE_FP32 = 1 } flce_dtype_t;
typedef enum {
  FLCE_MX_NONE = -1,
  FLCE_MXFP4 = 0,
  FLCE_MXFP8 = 1,
  FLCE_MXINT8 = 2
} flce_mx_format_t;

/* Bytes of a row of codes and of a row of scales for `cols` elements (either output may be
 * NULL).  1 <= cols <= 2^20. */
flce_status_t flce_mx_sizes(int64_t cols, int format, int64_t* code_bytes, int64_t* scale_bytes);

/*
 * Quantise x [rows, cols] (bf16 or fp32, ldx elements between rows) to codes and scales, or
 * write the values they stand for to out (rounded to nearest; every value of the three
 * formats is exact in bf16 and fp32 unless its scale is near the end of the type's range).
 * 0 <= rows <= 2^30; codes and scales 16-byte aligned; x and out naturally aligned, with
 * any row stride >= cols.
 */
flce_status_t flce_mx_quantize(const void* x, int x_dtype, int64_t ldx, int64_t rows, int64_t cols,
                               int format, void* codes, void* scales,
                               struct ihipStream_t* stream);
flce_status_t flce_mx_dequantize(const void* codes, const void* scales, int format, int64_t rows,
                                 int64_t cols, void* out, int out_dtype, int64_t ldo,
                                 struct ihipStream_t* stream);

/*
 * Layer norm over the rows of x [M, H], in 32 bits:
 *   mean = sum x / H,  rstd = 1 / sqrt(sum (x - mean)^2 / H + eps)
 *   y = weight (x - mean) rstd + bias          (NULL weight: 1, NULL bias: 0)
 * x and y are (bf16, bf16), (fp32, bf16) or (fp32, fp32); weight and bias bf16 or fp32;
 * mean and rstd fp32 [M].  With a checkpoint format (FLCE_MXFP8 or FLCE_MXINT8; otherwise
 * FLCE_MX_NONE) the call also writes x in that format to codes and scales, for a backward
 * that keeps a quarter to a half of x's bytes; y, mean and rstd are those of x itself.
 * 0 <= M <= 2^30 (0: nothing is touched), 1 <= H <= 2^20; any row strides >= H (rows of
 * multiples of 8 elements at 16-byte aligned addresses move fastest).  y may be x where
 * their types and strides agree.
 */
flce_status_t flce_layer_norm_forward(const void* x, int x_dtype, int64_t ldx, const void* weight,
                                      const void* bias, int param_dtype, int64_t M, int64_t H,
                                      float eps, void* y, int y_dtype, int64_t ldy, float* mean,
                                      float* rstd, int format, void* codes, void* scales,
                                      struct ihipStream_t* stream);

/* Workspace bytes of flce_layer_norm_backward (the partial sums of dweight and dbias). */
flce_status_t flce_layer_norm_backward_workspace(int64_t M, int64_t H, size_t* bytes);

/*
 * Backward of the layer norm, with xh = (x - mean) rstd from the forward's mean and rstd:
 *   g = weight dy,  dx = rstd (g - mean_j g - xh mean_j(g xh))
 *   dweight = sum_m dy xh,  dbias = sum_m dy       (param_dtype; either may be NULL)
 * x is given either itself (format FLCE_MX_NONE; dx has its type) or, with x NULL, as the
 * forward's checkpoint (format, codes, scales; dx bf16 or fp32).  dy is bf16 or fp32 (fp32
 * only with fp32 dx).  M = 0 writes zeros to dweight and dbias.  The sums over rows are
 * formed in a fixed order without atomics: results are bitwise repeatable.  workspace:
 * 256-byte aligned, at least flce_layer_norm_backward_workspace bytes.  dx may be dy or x
 * where their types and strides agree.
 */
flce_status_t flce_layer_norm_backward(const void* dy, int dy_dtype, int64_t lddy, const void* x,
                                       int x_dtype, int64_t ldx, int format, const void* codes,
                                       const void* scales, const void* weight, int param_dtype,
                                       const float* mean, const float* rstd, int64_t M, int64_t H,
                                       void* dx, int dx_dtype, int64_t lddx, void* dweight,
                                       void* dbias, void* workspace, size_t workspace_bytes,
                                       struct ihipStream_t* stream);

/*
 * The head with 4-bit weights: W [V, H] as FLCE_MXFP4 codes and scales from
 * flce_mx_quantize, for sampling from a compressed head (logits) and for scoring with a
 * frozen reference model (log-probs).  X [M, H] bf16 is rounded to MXFP4 on the way, so
 *   z[m, v] = scale * sum_k Q(X)[m, k] W[v, k]
 * with exact products and fp32 accumulation, in an order that depends on the shape of the
 * call (never on the workspace).  Shapes as in flce_workspace_query; X and both parts of W
 * 16-byte aligned; a vocabulary shard is a slice of W's rows.  A row of X that holds an
 * infinity or a NaN gives NaNs in its own outputs, a block of W that stands for NaNs gives
 * them in its column of the logits and in every row's logprob, lse and entropy (logprob and
 * entropy of an ignored row stay 0).  Errors of logprob, lse and entropy are relative to the
 * row's largest |z|; past |z| = 2^30 a row may come out as NaN, here and in flce_forward.
 *
 * flce_mx_logits writes z to out [M, V] (bf16 or fp32, any row stride >= V, naturally
 * aligned).  flce_mx_forward writes logprob, lse and entropy of targets, which never leave
 * the chip as logits: validity, ignored rows, outputs and token waves as in flce_forward,
 * with z from the 4-bit operands.  Workspaces: 256-byte aligned; flce_mx_workspace_query
 * gives what flce_mx_logits needs and what flce_mx_forward takes all rows at once with (a
 * smaller one, down to one wave of 256 rows, runs in waves; for large calls both hold a copy
 * of W's scale bytes in another order).  M = 0 is accepted and touches nothing.  Not differentiable: the weights are frozen.
 */
flce_status_t flce_mx_workspace_query(int64_t M, int64_t H, int64_t V, int compute_entropy,
                                      size_t* logits_bytes, size_t* fwd_bytes);
flce_status_t flce_mx_logits(const void* X, const void* W_codes, const void* W_scales, int64_t M,
                             int64_t H, int64_t V, float scale, void* out, int out_dtype,
                             int64_t ldo, void* workspace, size_t workspace_bytes,
                             struct ihipStream_t* stream);
flce_status_t flce_mx_forward(const void* X, const void* W_codes, const void* W_scales,
                              const int64_t* targets, int64_t M, int64_t H, int64_t V,
                              int64_t ignore_index, float scale, int compute_entropy,
                              float* logprob, float* lse, float* entropy, void* workspace,
                              size_t workspace_bytes, struct ihipStream_t* stream);

/*
 * Matrix product with bias, activation and residual in its epilogue: the dense block in front of
 * a head, or a head's logits.
 *   pre = X W^T + bias,  out = act(pre) + residual       (NULL bias, residual: none)
 * X [M, K] and W [N, K] bf16, products exact, sums in fp32; bias [N], residual and out [M, N]
 * bf16 or fp32, pre bf16 (NULL: not written).  Activations: none, relu, gelu (x Phi(x)),
 * gelu_tanh (x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) / 2), silu (x / (1 + e^-x)).
 * 0 <= M <= 2^30 (0: nothing is touched), 1 <= N <= 2^20, K a multiple of 8 up to 2^20.  Rows of
 * X and W are 16-byte aligned, with row strides (elements) up to 2^21; the other matrices are
 * naturally aligned with any row strides >= N (rows of multiples of 8 elements at 16-byte aligned
 * addresses move fastest).  out may be residual where their types and strides agree (otherwise the
 * call is refused).  workspace: 256-byte aligned, at least the forward bytes of
 * flce_linear_workspace (0: may be NULL).  Results are bitwise repeatable; the order of summation
 * depends on the shape.
 */
typedef enum {
  FLCE_ACT_NONE = 0,
  FLCE_ACT_RELU = 1,
  FLCE_ACT_GELU = 2,
  FLCE_ACT_GELU_TANH = 3,
  FLCE_ACT_SILU = 4
} flce_activation_t;

/*
 * Workspace bytes of flce_linear_forward and flce_linear_backward (either output may be NULL).  Sizes
 * whose tiles do not fit a launch (results of half a terabyte and more) are refused here as in the call
 * (the backward's: with every gradient wanted).
 */
flce_status_t flce_linear_workspace(int64_t M, int64_t N, int64_t K, size_t* fwd_bytes,
                                    size_t* bwd_bytes);
flce_status_t flce_linear_forward(const void* X, int64_t ldx, const void* W, int64_t ldw,
                                  const void* bias, int bias_dtype, int activation,
                                  const void* residual, int residual_dtype, int64_t ldr, int64_t M,
                                  int64_t N, int64_t K, void* out, int out_dtype, int64_t ldo,
                                  void* pre, int64_t ldp, void* workspace, size_t workspace_bytes,
                                  struct ihipStream_t* stream);

/*
 * Backward of it, from the forward's pre (unused without an activation; relu's slope at 0 is 0):
 *   dpre = dy act'(pre),  dX = dpre W,  dW = dpre^T X,  dbias = sum_m dpre
 * (the residual's gradient is dy itself).  dy bf16 or fp32; dX [M, K] and dW [N, K] bf16 with any
 * row strides; dbias [N] bf16 or fp32; each may be NULL.  dpre is rounded to bf16 for dW and dX
 * (the operands of the matrix instruction), not for dbias nor for a dX of M K <= 1024 values, over
 * which the roundings do not average out.  X is needed for dW, W for dX.  M = 0 writes zeros to dW and dbias.  No atomics: bitwise repeatable.  workspace as above,
 * with the backward bytes.
 */
flce_status_t flce_linear_backward(const void* dy, int dy_dtype, int64_t lddy, const void* pre,
                                   int64_t ldp, int activation, const void* X, int64_t ldx,
                                   const void* W, int64_t ldw, int64_t M, int64_t N, int64_t K,
                                   void* dX, int64_t lddx, void* dW, int64_t lddw, void* dbias,
                                   int bias_dtype, void* workspace, size_t workspace_bytes,
                                   struct ihipStream_t* stream);

/*
 * Dropout over x [M, H] and the residual it is added to (NULL: none):
 *   y = residual + x keep / (1 - q),  keep[m, h] = bits[m, h] >= threshold
 * with threshold = 65536 p rounded to nearest, q = threshold / 65536, and 16 random bits an
 * element from Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC11): counter (h / 8, m, offset low,
 * offset high), key (seed low, seed high); column h takes word (h % 8) / 2, the low half where h
 * is even.  The mask is not stored: the gradient of x is the same call on dy without a residual
 * (the residual's gradient is dy itself).  seed_at (NULL: seed counts) is a place in device memory
 * that the kernel reads the seed from, so that a captured call draws anew where its caller writes
 * there.  A call needs a (seed, offset) of its own for masks of its own.  x, residual and y are
 * bf16 or fp32 each, with any row strides, naturally aligned; 0 <= p <= 1 (1: everything is
 * dropped); sums in fp32; a dropped infinity or NaN is gone.  0 <= M <= 2^30 (0: nothing is
 * touched), 1 <= H <= 2^20.  y may be x or residual where their types and strides agree (otherwise
 * the call is refused).
 */
flce_status_t flce_dropout(const void* x, int x_dtype, int64_t ldx, const void* residual,
                           int residual_dtype, int64_t ldr, int64_t M, int64_t H, double p,
                           uint64_t seed, const uint64_t* seed_at, uint64_t offset, void* y,
                           int y_dtype, int64_t ldy, struct ihipStream_t* stream);

/*
 * Log-probs of given tokens, entropy and the largest alternatives from logits x [M, V] (bf16 or
 * fp32, any row stride, naturally aligned), under softmax(scale x), 0 < scale <= 2^64:
 *   logprob[m, j] = log p[m, tokens[m, j]]     (0 where the token is ignore_index or outside
 *                                               [0, V); tokens int64 [M, n_tokens])
 *   lse[m] = log sum_v exp(scale x),  entropy[m] = -sum_v p log p          (NULL: not wanted)
 *   top_ids[m, i], top_logprob[m, i]: the n_top largest logits of the row, in falling order,
 *                                     equal ones by their index
 * and stats[m] = (largest logit, log sum_v exp(scale (x - largest))) for the backward.  All of
 * them fp32, ids int64; sums in fp32.  A logit of -inf is masked: it has probability 0 and adds
 * nothing.  In a row that is masked throughout lse and every log-prob are -inf and entropy is 0.
 * In a row with a NaN or +inf they are NaN, the alternatives in their order all the same, NaNs
 * with the masked ones.  0 <= M <= 2^30 (0: nothing is touched), 1 <= V <= 2^30, n_tokens <=
 * FLCE_MAX_TOKENS, n_top <= FLCE_MAX_TOP and V; either may be 0.  workspace: 256-byte aligned, at
 * least flce_token_logprobs_workspace bytes (0: may be NULL).
 */
#define FLCE_MAX_TOP 128
#define FLCE_MAX_TOKENS 1024
flce_status_t flce_token_logprobs_workspace(int64_t M, int64_t V, int64_t n_top, size_t* bytes);
flce_status_t flce_token_logprobs(const void* logits, int dtype, int64_t ldl, int64_t M, int64_t V,
                                  const int64_t* tokens, int64_t n_tokens, int64_t ignore_index,
                                  float scale, int64_t n_top, float* logprob, float* lse,
                                  float* entropy, float* stats, int64_t* top_ids,
                                  float* top_logprob, void* workspace, size_t workspace_bytes,
                                  struct ihipStream_t* stream);

/*
 * Gradient of those with respect to the logits:
 *   dx[m, v] = scale (sum_j g[m, j] (1[v = t[m, j]] - p[m, v])
 *                     - b[m] p[m, v] (log p[m, v] + entropy[m]) + c[m] p[m, v])
 * over the given tokens with grad_logprob [M, n_tokens] and the alternatives with grad_top [M,
 * n_top] (NULL: none of them), b = grad_entropy [M] (NULL: 0; needs the forward's entropy), c =
 * grad_lse [M] (NULL: 0).  The terms with p are 0 where p is 0 in fp32, at any scale and b.  Ignored
 * and invalid tokens add nothing; a token given several times adds each of its gradients.  dlogits
 * has the logits' type, any row stride, and may be their own memory.  Rows that nothing valid is
 * asked of, and rows masked throughout, get zeros; a NaN gradient reaches every element of its row.
 */
flce_status_t flce_token_logprobs_backward(const void* logits, int dtype, int64_t ldl, int64_t M,
                                           int64_t V, const int64_t* tokens, int64_t n_tokens,
                                           int64_t ignore_index, float scale, const float* stats,
                                           const float* entropy, const int64_t* top_ids,
                                           int64_t n_top, const float* grad_logprob,
                                           const float* grad_top, const float* grad_entropy,
                                           const float* grad_lse, void* dlogits, int64_t ldd,
                                           struct ihipStream_t* stream);

/* Static description of a status code. */
const char* flce_status_string(flce_status_t status);

/* Thread-local detail of the last failure on this thread ("" if none). */
const char* flce_last_error_message(void);

/* Library version as "major.minor.patch". */
const char* flce_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LIBFLCE_FLCE_H */
