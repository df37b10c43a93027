/*
 * dgt_experts.h -- C interface of the operators around a mixture-of-experts
 * feed-forward block on GB300 (sm_103a), in the same library as dgt_gemm.h.
 *
 * The block, for T tokens of hidden size H, E experts and k experts a token:
 *
 *   h, y      = gemm_rmsnorm            h = x + residual, y = norm(h) * weight (16-bit, or E4M3 rows with scales)
 *   ids, ...  = gemm_route              which experts a token goes to, with what weights, and the expert order:
 *                                       the T * k (token, expert) pairs sorted by expert
 *   c         = gemm_*_grouped          each expert's rows times its weight matrix, one launch for all experts
 *   out       = gemm_combine            each token's weighted sum over its k rows (and a residual)
 *
 * with gemm_rmsnorm_backward, gemm_route_backward, gemm_*_grouped (with the
 * other layout flag) and gemm_*_grouped_wgrad, and gemm_combine_backward as
 * their gradients. The GEMM pages have no counterpart to these calls.
 *
 * Common rules, as in dgt_gemm.h: every pointer is device (or managed) memory
 * of the current device and is the caller's; a call enqueues its work on
 * `stream` and returns at once; the return value is a GEMM_* code that reports
 * argument and launch errors; nothing is allocated (a call that needs scratch
 * takes a workspace, whose size a *_workspace call gives); results are
 * deterministic run to run (no floating-point atomics); the calls are safe
 * from several host threads and may be captured in a CUDA graph. Leading
 * dimensions are in elements; an element type's values are aligned to its
 * size. Sums, softmax statistics and norms are held in fp32. Outputs must not
 * overlap inputs except where a call says so.
 *
 * Expert order: slot s of [0, offsets[E]) holds one (token, expert) pair;
 * expert e owns slots offsets[e] .. offsets[e+1]-1; within an expert the
 * slots follow (token, choice) order. offsets, row and slot numbers are read
 * on the device: the calls clamp what lies outside the stated ranges, so a
 * wrong one gives a wrong result and never an access outside the buffers.
 */
#ifndef DGT_EXPERTS_H
#define DGT_EXPERTS_H

#include "dgt_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types (the `kind` numbers of gemm_plan_query). */
#define GEMM_TYPE_F16 0
#define GEMM_TYPE_BF16 1
#define GEMM_TYPE_F32 2
#define GEMM_TYPE_E4M3 3

/*
 * Root-mean-square norm of `rows` rows of `cols` elements, with the residual's
 * addition and an optional 8-bit output:
 *   h    = x + residual, rounded to `type` (x itself when residual is NULL)
 *   r    = 1 / sqrt(mean_j(h[j]^2) + eps)             (fp32; of the rounded h)
 *   y[j] = h[j] * r * weight[j], rounded once to y_type
 * type: F16, BF16 or F32 (x, residual, weight, h); y_type: the same, or E4M3,
 * which gives q[j] = e4m3(y[j] * (1 / s)) (round to nearest even) and the
 * row's scale s = max(max_j |y[j]|, 1e-12) / 448 in y_scale[row], so that
 * q * s stands for y; a NaN in a row makes its scale NaN. y_scale must be NULL
 * for the other types. h (written only with a residual; may be NULL, or the
 * very buffer and pitch of x or of residual) and rstd (r of each row) may be
 * NULL. y may be the very buffer and pitch of x where their types are the same.
 * cols <= 16384; with no rows or no columns nothing is written.
 */
int gemm_rmsnorm(int type, int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                 const void* weight, float eps, void* h, int64_t ldh, int y_type, void* y, int64_t ldy,
                 float* y_scale, float* rstd, void* stream);

/*
 * Its gradient: from dy (of y before any 8-bit rounding), h, weight and rstd,
 *   g = dy * weight, xhat = h * rstd
 *   dx[j] = rstd * (g[j] - xhat[j] * mean_i(g[i] * xhat[i])) + dh[j]
 *   dw[j] = sum over rows of dy[j] * xhat[j]
 * dh, the gradient that reaches h by the residual path, may be NULL; dx is the
 * gradient of both x and residual (and may be the very buffer and pitch of dh
 * or dy); dw has the weight's type. workspace: gemm_rmsnorm_backward_workspace
 * bytes, 16-byte aligned, for the row blocks' partial sums of dw, which are
 * added in a fixed order.
 */
int gemm_rmsnorm_backward(int type, int64_t rows, int64_t cols, const void* dy, int64_t lddy, const void* h,
                          int64_t ldh, const void* weight, const float* rstd, const void* dh, int64_t lddh, void* dx,
                          int64_t lddx, void* dw, void* workspace, int64_t workspace_bytes, void* stream);
int64_t gemm_rmsnorm_backward_workspace(int64_t rows, int64_t cols);

/* Router scores */
#define GEMM_SCORE_SOFTMAX 0
#define GEMM_SCORE_SIGMOID 1

/*
 * How gemm_route chooses. For a token with logits l:
 *   score[e] = softmax(l)[e], or sigmoid(l[e])
 *   key[e]   = score[e] + bias[e] (bias only moves the choice, not the weights)
 *   with groups > 1 the experts form that many equal runs; a group's key is
 *   the sum of its two largest keys (its only one if it has one), and only
 *   experts of the kept_groups best groups stay
 *   ids      = the k experts of largest key, in descending order
 *   weight   = score[id], divided by (the chosen scores' sum + 1e-20) if renormalize != 0, times `scale`
 * Equal keys, and equal group keys, go to the lowest index. A logit of -inf
 * takes its expert out: it is never chosen; where fewer than k experts are
 * left the remaining ids are -1, with weight 0 and no slot. An expert whose
 * score is NaN is never chosen, and makes all the token's weights NaN (with
 * softmax one NaN or +inf logit does that to every expert of the token).
 */
typedef struct gemm_route_config {
  int k;
  int score;
  int groups;
  int kept_groups;
  int renormalize;
  float scale;
} gemm_route_config_t;

/*
 * Routing of `tokens` rows of `experts` logits (F16, BF16 or F32; leading
 * dimension ld) and the expert order. Outputs: ids and weights (tokens x k),
 * slots (tokens x k: each pair's place in the expert order, -1 for id -1),
 * rows (tokens * k: the token of each slot; -1 past offsets[experts]), offsets
 * (experts + 1). bias: `experts` floats or NULL. 1 <= experts <= 1024, 1 <= k <=
 * 32, k <= kept_groups * experts / groups, tokens * k < 2^31. The softmax
 * denominator is summed by adding halves (x[i] + x[i + n/2], n a power of two,
 * zero padded, down to one value), so equal logits give equal keys whatever
 * kernel runs. workspace: gemm_route_workspace bytes (may be 0), 16-byte aligned.
 */
int gemm_route(int type, int64_t tokens, int experts, const void* logits, int64_t ld, const float* bias,
               const gemm_route_config_t* config, int32_t* ids, float* weights, int32_t* slots, int32_t* rows,
               int32_t* offsets, void* workspace, int64_t workspace_bytes, void* stream);
int64_t gemm_route_workspace(int64_t tokens, int experts, int k);

/*
 * Gradient of the weights with respect to the logits (the choice is held
 * fixed): dlogits (tokens x experts, the logits' type, fully written) from
 * dweights (tokens x k), the logits and ids. Pairs with id -1 are skipped.
 * config: score, renormalize, scale and k are used.
 */
int gemm_route_backward(int type, int64_t tokens, int experts, const void* logits, int64_t ld, const int32_t* ids,
                        const float* dweights, const gemm_route_config_t* config, void* dlogits, int64_t ldd,
                        void* stream);

/* Activation of the grouped products beyond GEMM_ACT_NONE .. GEMM_ACT_GELU_TANH:
 * W holds gate columns [0, N/2) and value columns [N/2, N), N even, and
 * C[s][j] = g / (1 + exp(-g)) * v has N/2 columns. */
#define GEMM_ACT_SILU_GATED 4

/*
 * Epilogue of a grouped product, in fp32 from the fp32 accumulator, rounded
 * once: act(alpha * row_scale[row(s)] * col_scale[e][j] * acc + bias[e][j]).
 * row_scale: one per row of A; col_scale: `groups` x N; bias: groups x N of
 * C's type; each may be NULL. GEMM_ACT_GELU_TANH and the gated SiLU take the
 * hardware's exponential: within 4e-5 of their values before the rounding, and 0
 * where 1 + exp passes 2^126 (gates below -87.3). The dense calls' tanh form is another.
 */
typedef struct gemm_grouped_epilogue {
  float alpha;
  const float* row_scale;
  const float* col_scale;
  const void* bias;
  int activation;
} gemm_grouped_epilogue_t;

/*
 * Grouped product: for each group e (expert) and slot s in
 * [offsets[e], offsets[e+1]),
 *   C[s] = epilogue(A[row(s)] . W_e),   row(s) = rows ? rows[s] : s
 * A: a_rows x K, row-major. W_e starts e * stride_w elements after W_0:
 * layout GEMM_B_ROW_MAJOR K x N, GEMM_B_K_MAJOR N x K (E4M3: this one only).
 * C: slots x N (N/2 for GEMM_ACT_SILU_GATED); F16 and BF16 keep their type,
 * E4M3 gives BF16. offsets: groups + 1 numbers on the device, offsets[0] = 0,
 * not decreasing, the last at most `slots`; C's rows from offsets[groups] to
 * `slots` are set to zero. `rows` NULL needs a_rows >= slots. With the other
 * layout flag the same call is the gradient of A: dA = dC . W_e^T, one row a
 * slot. epilogue NULL: C = A . W. 1 <= groups <= 1024; slots, N, K < 2^31;
 * K = 0 gives the epilogue of 0 (an A of no rows takes no row_scale then). A and
 * W must start on 16-byte boundaries (GEMM_ERR_MISALIGNED otherwise); C may have
 * any alignment that keeps its elements aligned.
 *
 * workspace: 128-byte aligned, gemm_grouped_rows_workspace + gemm_grouped_weights_workspace
 * bytes. The first are for A's rows, put in slot order before the product: rows of
 * a pitch that is not a multiple of 16 bytes (an A of one row may have any pitch),
 * and with `rows` those of groups that have many rows on average; without room
 * for them named rows are gathered on the way to shared memory (the same
 * results; slower where groups have many rows). The second are for a copy of W, made in
 * every call, where its pitch (of a W_e of more than one row) or its matrix
 * stride is not a multiple of 16 bytes, or where the second half of row-major
 * gated weights does not start on one: weights kept without these cost
 * nothing more. GEMM_ERR_MISALIGNED where a copy is needed and there is no room for
 * it. gemm_grouped_workspace: the first for A with rows of 16-byte multiples and `rows`.
 */
int64_t gemm_grouped_rows_workspace(int type, int groups, int64_t slots, int64_t K, int64_t a_rows, int64_t lda,
                                    int gathered);
int64_t gemm_grouped_weights_workspace(int type, int groups, int64_t N, int64_t K, int64_t ldw, int64_t stride_w,
                                       int layout, int activation);
int64_t gemm_grouped_workspace(int type, int groups, int64_t slots, int64_t K);
int gemm_f16_grouped(int groups, const int32_t* offsets, int64_t slots, int64_t N, int64_t K, const uint16_t* A,
                     int64_t a_rows, int64_t lda, const int32_t* rows, const uint16_t* W, int64_t ldw,
                     int64_t stride_w, uint16_t* C, int64_t ldc, int layout, const gemm_grouped_epilogue_t* epilogue,
                     void* workspace, int64_t workspace_bytes, void* stream);
int gemm_bf16_grouped(int groups, const int32_t* offsets, int64_t slots, int64_t N, int64_t K, const uint16_t* A,
                      int64_t a_rows, int64_t lda, const int32_t* rows, const uint16_t* W, int64_t ldw,
                      int64_t stride_w, uint16_t* C, int64_t ldc, int layout, const gemm_grouped_epilogue_t* epilogue,
                      void* workspace, int64_t workspace_bytes, void* stream);
int gemm_e4m3_grouped(int groups, const int32_t* offsets, int64_t slots, int64_t N, int64_t K, const uint8_t* A,
                      int64_t a_rows, int64_t lda, const int32_t* rows, const uint8_t* W, int64_t ldw,
                      int64_t stride_w, uint16_t* C, int64_t ldc, int layout, const gemm_grouped_epilogue_t* epilogue,
                      void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Gradient of the grouped product's weights:
 *   layout GEMM_B_K_MAJOR:   dW_e (N x K) = sum over the group's s of dC[s]^T A[row(s)]
 *   layout GEMM_B_ROW_MAJOR: dW_e (K x N) = sum over the group's s of A[row(s)]^T dC[s]
 * in fp32, rounded once to the operands' type; a group without slots gets
 * zeros. dC: slots x N. A, rows and dC as above (from 16-byte boundaries); dW
 * may have any alignment that keeps its elements aligned, stride_dw at least
 * one matrix's extent. workspace: gemm_grouped_wgrad_rows_workspace bytes
 * (`gathered`: `rows` is given), 128-byte aligned, for the groups' last, partly
 * filled slabs, for A's rows in slot order with `rows` or a pitch that is not a
 * multiple of 16 bytes, and for dC's rows with such a pitch.
 * gemm_grouped_wgrad_workspace: the same for pitches that are.
 */
int64_t gemm_grouped_wgrad_rows_workspace(int groups, int64_t slots, int64_t N, int64_t K, int64_t a_rows, int64_t lda,
                                          int gathered, int64_t lddc);
int64_t gemm_grouped_wgrad_workspace(int groups, int64_t slots, int64_t N, int64_t K, int gathered);
int gemm_f16_grouped_wgrad(int groups, const int32_t* offsets, int64_t slots, int64_t N, int64_t K, const uint16_t* A,
                           int64_t a_rows, int64_t lda, const int32_t* rows, const uint16_t* dC, int64_t lddc,
                           uint16_t* dW, int64_t lddw, int64_t stride_dw, int layout, void* workspace,
                           int64_t workspace_bytes, void* stream);
int gemm_bf16_grouped_wgrad(int groups, const int32_t* offsets, int64_t slots, int64_t N, int64_t K,
                            const uint16_t* A, int64_t a_rows, int64_t lda, const int32_t* rows, const uint16_t* dC,
                            int64_t lddc, uint16_t* dW, int64_t lddw, int64_t stride_dw, int layout, void* workspace,
                            int64_t workspace_bytes, void* stream);

/*
 * Weighted sum over a token's slots:
 *   y[t] = residual[t] + sum_j weights[t][j] * z[slots[t][j]]
 * z: nslots x cols; slots and weights tokens x k (a slot outside [0, nslots)
 * adds 0 times its weight: nothing, or NaN where that is not finite; weights NULL:
 * all 1); residual may be NULL or the very buffer and pitch of y. type F16, BF16 or F32 (z, residual, y); fp32
 * sums in the order of j, the residual last. 1 <= k <= 32.
 */
int gemm_combine(int type, int64_t tokens, int64_t cols, int k, const void* z, int64_t ldz, int64_t nslots,
                 const int32_t* slots, const float* weights, const void* residual, int64_t ldr, void* y, int64_t ldy,
                 void* stream);

/*
 * Its gradient: dz[slots[t][j]] = weights[t][j] * dy[t] (weights NULL: 1),
 * rows of dz from *used to nslots are set to zero (used: one number on the
 * device, offsets + experts of the expert order; NULL: none), dweights[t][j]
 * = dy[t] . z[slots[t][j]] in fp32 (0 for a slot outside [0, nslots));
 * dweights may be NULL (then z may be too). The slots must be distinct.
 */
int gemm_combine_backward(int type, int64_t tokens, int64_t cols, int k, const void* dy, int64_t lddy, const void* z,
                          int64_t ldz, int64_t nslots, const int32_t* slots, const float* weights,
                          const int32_t* used, void* dz, int64_t lddz, float* dweights, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DGT_EXPERTS_H */
