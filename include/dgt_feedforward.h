/*
 * dgt_feedforward.h -- C interface of the operators of a dense feed-forward
 * block on GB300 (sm_103a), in the same library as dgt_gemm.h and
 * dgt_experts.h:
 *
 *   gemm_layernorm        h = x + residual, y = (h - mean) / deviation * weight + bias (16-bit or FP32, or E4M3 rows)
 *   gemm_gated            act(A . gate) * (A . value), both products and the activation in one kernel
 *   gemm_e4m3_blocks      a product of E4M3 matrices with a scale for each block of 128
 *   gemm_quantize_blocks  16-bit or FP32 matrices in that form
 *
 * with gemm_layernorm_backward and gemm_gated_backward. The gradients of
 * gemm_e4m3_blocks are the same call on operands quantised along the other
 * dimension (gemm_quantize_blocks with `transpose`). The GEMM pages have no
 * counterpart to these calls.
 *
 * The common rules are dgt_experts.h's: device memory of the current device,
 * the caller's; work is enqueued on `stream` and the call returns at once; a
 * GEMM_* code; nothing is allocated; results are the same from run to run;
 * safe from several host threads, and capturable in a CUDA graph. Leading
 * dimensions are in elements. Sums and statistics are held in fp32. Outputs
 * must not overlap inputs, or each other, except where a call says so. Element
 * types are GEMM_TYPE_*.
 */
#ifndef DGT_FEEDFORWARD_H
#define DGT_FEEDFORWARD_H

#include "dgt_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Layer norm of `rows` rows of `cols` elements, with the residual's addition
 * and an optional 8-bit output:
 *   h    = x + residual, rounded to `type` (x itself when residual is NULL)
 *   m    = mean_j(h[j]),  r = 1 / sqrt(mean_j((h[j] - m)^2) + eps)      (fp32; of the rounded h)
 *   y[j] = (h[j] - m) * r * weight[j] + bias[j], rounded once to y_type
 * type: F16, BF16 or F32 (x, residual, weight, bias, h); y_type: the same, or
 * E4M3, which gives q[j] = e4m3(y[j] * (1 / s)) (round to nearest even) and the
 * row's scale s = max(max_j |y[j]|, 1e-12) / 448 in y_scale[row], so that
 * q * s stands for y; a NaN in a row makes its scale NaN. y_scale must be NULL
 * for the other types. bias, mean (m of each row) and rstd (r) may be NULL. h
 * (written only with a residual; may be NULL, or the very buffer and pitch of x
 * or of residual). y may be the very buffer and pitch of x where their types
 * are the same. cols <= 16384; with no rows or no columns nothing is written.
 */
int gemm_layernorm(int type, int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                   const void* weight, const void* bias, float eps, void* h, int64_t ldh, int y_type, void* y,
                   int64_t ldy, float* y_scale, float* mean, float* rstd, void* stream);

/*
 * Its gradient: from dy (of y before any 8-bit rounding), h, weight, mean and rstd,
 *   xhat = (h - mean) * rstd, g = dy * weight
 *   dx[j] = rstd * (g[j] - mean_i(g[i]) - xhat[j] * mean_i(g[i] * xhat[i])) + dh[j]
 *   dw[j] = sum over rows of dy[j] * xhat[j],  db[j] = sum over rows of dy[j]
 * dh, the gradient that reaches h by the residual path, may be NULL, and so may
 * db; dx is the gradient of both x and residual (and may be the very buffer and
 * pitch of dh or dy); dw and db have the weight's type. workspace:
 * gemm_layernorm_backward_workspace bytes, 16-byte aligned, for the row blocks'
 * partial sums, which are added in a fixed order.
 */
int gemm_layernorm_backward(int type, int64_t rows, int64_t cols, const void* dy, int64_t lddy, const void* h,
                            int64_t ldh, const void* weight, const float* mean, const float* rstd, const void* dh,
                            int64_t lddh, void* dx, int64_t lddx, void* dw, void* db, void* workspace,
                            int64_t workspace_bytes, void* stream);
int64_t gemm_layernorm_backward_workspace(int64_t rows, int64_t cols);

/* Activation of a gated product's gate half. */
#define GEMM_GATE_SILU 0
#define GEMM_GATE_GELU 1
#define GEMM_GATE_GELU_TANH 2
#define GEMM_GATE_RELU 3

/*
 * Gated product: with up = A . W + bias (M x 2F, fp32),
 *   C[i][j] = act(up[i][j]) * up[i][F + j]          (M x F, rounded once)
 * type: F16 or BF16 (A, W, bias, C, up). A: M x K, row-major. W holds the gate
 * columns [0, F), then the value columns [F, 2F): layout GEMM_B_ROW_MAJOR
 * K x 2F, GEMM_B_K_MAJOR 2F x K. bias: 2F elements or NULL. `up` (M x 2F, or
 * NULL) receives the rounded sums that gemm_gated_backward takes; C is computed
 * from the fp32 ones. SiLU and GELU's tanh form take the hardware's exponential:
 * within 4e-5 of their values before the rounding, and 0 where 1 + exp passes
 * 2^126 (gates below -87.3). GELU's other form is 1 + erf in fp32: within 2e-7 of
 * the gate's size, which leaves few digits of its tail below about -4. M, 2F, K < 2^31; K = 0 gives the products of no
 * terms. A and W start on 16-byte boundaries (GEMM_ERR_MISALIGNED otherwise); C
 * and up may have any alignment that keeps their elements aligned.
 * workspace: gemm_gated_workspace bytes (0 for most), 128-byte aligned: where
 * the pitch of A or W is not a multiple of 16 bytes, or the value half of
 * row-major weights does not start on one, they are copied there first, in
 * every call. A few rows take a kernel of their own only where A and W are read in
 * place; it adds up in another order, so that the same numbers at another pitch may
 * give another last bit.
 */
int gemm_gated(int type, int64_t M, int64_t F, int64_t K, const void* A, int64_t lda, const void* W, int64_t ldw,
               int layout, int activation, const void* bias, void* C, int64_t ldc, void* up, int64_t ldup,
               void* workspace, int64_t workspace_bytes, void* stream);
int64_t gemm_gated_workspace(int type, int64_t M, int64_t F, int64_t K, int64_t lda, int64_t ldw, int layout);

/*
 * Its gradient, from dC (M x F), up (M x 2F, as gemm_gated kept it), A and W:
 *   dup[i][j] = dC[i][j] * up[i][F + j] * act'(up[i][j]),  dup[i][F + j] = dC[i][j] * act(up[i][j])
 *   dA = dup . W^T (M x K),  dW = A^T . dup (W's layout),  dbias[j] = sum over i of dup[i][j]
 * dup is rounded to `type` for the products (dbias sums it in fp32 before that);
 * the products are fp32 sums, rounded once. dA, dW and dbias may each be NULL; A
 * is read for dW only, W for dA only. act'(0) of ReLU is 0. dA, dW, dC and up
 * may have any alignment that keeps their elements aligned; A and W as above.
 * workspace: gemm_gated_backward_workspace bytes (want_*: which outputs are asked
 * for), 128-byte aligned: dup, and what the products stage.
 */
int gemm_gated_backward(int type, int64_t M, int64_t F, int64_t K, const void* dC, int64_t lddc, const void* up,
                        int64_t ldup, const void* A, int64_t lda, const void* W, int64_t ldw, int layout,
                        int activation, void* dA, int64_t ldda, void* dW, int64_t lddw, void* dbias, void* workspace,
                        int64_t workspace_bytes, void* stream);
int64_t gemm_gated_backward_workspace(int type, int64_t M, int64_t F, int64_t K, int64_t lda, int64_t ldw, int layout,
                                      int want_da, int want_dw, int want_dbias);

/*
 * Product of E4M3 matrices with a scale for each block of 128 along K:
 *   C[i][j] = sum over blocks b of a_scale[i][b] * b_scale[j][b] * (sum over k of block b of A[i][k] * B[j][k])
 * A: M x K, B: N x K (K-major), C: M x N BF16, rounded once from fp32. The sum of
 * a block is the tensor cores' fp32; blocks are scaled and added in fp32, in
 * order (where a few rows are split along K: each part in order, then the parts).
 * a_scale[i][b] is at a_scale[i * as_row + b * as_block], for b < ceil(K / 128).
 * b_scale: b_rows = 1 the same, with bs_row and bs_block; b_rows = 128 has a scale
 * for each 128 x 128 block, b_scale[(j / 128) * bs_row + b * bs_block]. Strides may be
 * 0 (a scale for a whole row). K = 0 gives zeros. A and B start on 16-byte
 * boundaries and their pitches are multiples of 16 (but for a matrix of one row):
 * GEMM_ERR_MISALIGNED otherwise. A scale that is not finite reaches the entries
 * that it belongs to, also where the block's sum is 0 (as NaN). A block's two
 * scales are multiplied with each other, then with its sum: their product has to
 * be within fp32's normal range, and each of them may be anywhere in it.
 */
int gemm_e4m3_blocks(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const float* a_scale,
                     int64_t as_row, int64_t as_block, const uint8_t* B, int64_t ldb, const float* b_scale,
                     int64_t bs_row, int64_t bs_block, int b_rows, uint16_t* C, int64_t ldc, void* stream);

/*
 * A matrix in that form. With transpose = 0, t = x; else t = x^T:
 *   s = max(max |t| over the block, 1e-12) / 448,  q = e4m3(t * (1 / s)), round to nearest even
 * for blocks of block_rows (1 or 128) rows of t x 128 columns of t, the last ones
 * smaller. x: rows x cols, F16, BF16 or F32. q has t's shape, ldq apart; bytes
 * between its rows are left as they were. scale[i][b] is at scale[i * s_row + b *
 * s_block], i counting t's rows (block_rows = 1) or runs of 128 of them. A NaN
 * makes its block's scale NaN; an infinity makes it infinite, and the block's
 * finite values 0.
 */
int gemm_quantize_blocks(int type, int64_t rows, int64_t cols, const void* x, int64_t ldx, int block_rows,
                         int transpose, uint8_t* q, int64_t ldq, float* scale, int64_t s_row, int64_t s_block,
                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DGT_FEEDFORWARD_H */
