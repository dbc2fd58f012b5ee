/*
 * mxfp4_train.h -- C ABI of libmxfp4_train.so: what a training step needs beside the FP4 linear
 * layers of mxfp4.h, for AMD MI355X (gfx950).
 *
 *  - 8-bit linear products (mxfp4_fp8_*): the three GEMMs of a linear layer in E4M3 with a
 *    power-of-two scale for each block of 128, for layers that FP4 is too coarse for;
 *  - the loss of the head (mxfp4_linear_xent_*): softmax cross entropy of a last linear layer over a
 *    large vocabulary, in pieces of it and without keeping the logits, and its gradients;
 *  - the orthogonalised update (mxfp4_orthogonalize): Newton-Schulz steps on a weight gradient, such
 *    as mxfp4_linear_wgrad writes.
 *
 * The library is a separate one, so that libmxfp4.so and its ABI version stay what they are.
 * Conventions are those of mxfp4.h: device pointers owned by the caller and only used until the
 * enqueued work ends; asynchronous on `stream`; argument errors found before any launch, nothing
 * launched and no output touched; workspaces given by the caller (256-byte aligned, in use until the
 * work ends: two calls, or two captured graphs, that may run at the same time need one each); no
 * state between calls; sizes that need more than a grid holds (2^32 work-items) are MXFP4_ERR_SHAPE, and
 * 0 to the workspace queries; results that do not change from run to run (no atomics); gfx950 only. Every
 * call can be captured into a graph.
 */
#ifndef MXFP4_TRAIN_H_
#define MXFP4_TRAIN_H_

#include "mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Raised whenever an entry point, an argument's meaning or a layout changes. */
#define MXFP4_TRAIN_ABI_VERSION 1

/* MXFP4_TRAIN_ABI_VERSION of the built library. */
int mxfp4_train_abi_version(void);

/* ---------------------------------------------------------------------------------------------
 * 8-bit linear products.
 *
 * A quantized operand with `outer` rows of length L has codes q[outer][ldq], E4M3 (sign, four
 * exponent bits of bias 7, three mantissa bits; OCP 8-bit floating point, no infinities, largest
 * value 448), and scales s[outer][lds], one E8M0 byte S (value 2^(S-127); 0xFF = NaN) for each 128
 * consecutive codes: value = code * 2^(S-127). A row holds round_up(L, 128) codes, those behind L
 * zero, and ceil(L / 128) scales.
 *
 * Scale: the smallest S >= 0 with amax <= 448 * 2^(S-127) over the block, so that nothing saturates;
 * 0 for a block of zeros; 0xFF and codes 0 for a block that holds a NaN or an infinity (its
 * products are then NaN). Code: x * 2^(127-S) (exact unless it is subnormal) rounded to nearest,
 * ties to even.
 *
 * Block: MXFP4_FP8_ROW, 1 x 128 along the quantized axis (activations, gradients), or
 * MXFP4_FP8_TILE, 128 x 128, the same byte in every row of the tile (weights: both axes' codes are
 * then the same numbers). Blocks are counted from the tensor's first row and column; the last
 * ones may be short.
 */
typedef enum { MXFP4_FP8_ROW = 0, MXFP4_FP8_TILE = 1, MXFP4_ENUM_RANGE(MXFP4_FP8_BLOCK) } mxfp4_fp8_block_t;

/*
 * mxfp4_fp8_quantize -- one or both quantizations of x[rows][cols] (row stride ldx elements) from one read.
 *   q1, ldq1, s1, lds1   along the rows (outer = rows, L = cols), or q1 = NULL;
 *   q0, ldq0, s0, lds0   along the columns, the quantized transpose (outer = cols, L = rows), or q0 = NULL.
 * Requirements: rows, cols >= 0; fewer than 2^24 tiles of 128 x 128; ldx >= cols; for each output
 * ldq >= round_up(L, 128) and a multiple of 16, q 16-byte aligned, lds >= ceil(L / 128). x needs its
 * element's alignment only (16 bytes, with 16-byte rows, are read faster). Nothing overlaps.
 */
mxfp4_status_t mxfp4_fp8_quantize(const void *x, mxfp4_dtype_t dtype, int64_t rows, int64_t cols, int64_t ldx,
                                  mxfp4_fp8_block_t block, uint8_t *q1, int64_t ldq1, uint8_t *s1, int64_t lds1,
                                  uint8_t *q0, int64_t ldq0, uint8_t *s0, int64_t lds0, void *stream);

/*
 * mxfp4_fp8_gemm -- c = alpha * A B^T + beta * c on the scaled FP8 matrix cores, FP32 accumulation.
 *   A = (aq [M][lda bytes], as [M][ldas]), B = (bq [N][ldb], bs [N][ldbs]), both of length K as above.
 *   c  FP32 or bf16 (rounded to nearest even once) [M][ldc], element-aligned; read only when beta != 0.
 * Requirements: M, N, K >= 0 and < 2^31; fewer than 2^23 tiles of 256 x 256 in c; lda, ldb >=
 * round_up(K, 128), multiples of 16, below 2^24; ldas, ldbs multiples of 16 with the scales' rows readable
 * in whole 16 bytes; all four operand pointers 16-byte aligned; ldc >= N. K == 0 gives beta * c. c overlaps
 * no operand.
 * Sums: the matrix cores add the products of eight consecutive codes at a time and first cut each, toward
 * zero, to a multiple of 2^-13 of the largest one's power of two; the sums of eight are added in FP32. On
 * Gaussian operands the result is off by 1.5e-5 of its norm, at worst by 7 * 2^-13 of the sum over
 * the groups of eight of their largest |product|. That holds for FP32 results too.
 * workspace (optional, 256-byte aligned, mxfp4_fp8_gemm_workspace_bytes() bytes): lets a product with
 * few output tiles split its contraction (added up in a fixed order); without it, it runs unsplit.
 */
mxfp4_status_t mxfp4_fp8_gemm(const uint8_t *aq, int64_t lda, const uint8_t *as, int64_t ldas, const uint8_t *bq,
                              int64_t ldb, const uint8_t *bs, int64_t ldbs, int64_t M, int64_t N, int64_t K, float alpha,
                              float beta, void *c, mxfp4_out_dtype_t c_dtype, int64_t ldc, void *workspace, size_t ws_bytes,
                              void *stream);
size_t mxfp4_fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * The three GEMMs of a linear layer Y = X W^T: both operands quantized in one launch, then multiplied.
 *   fprop: y[M][N]  = X[M][K] . W[N][K]^T    X in 1 x 128 blocks along K, W in 128 x 128
 *   dgrad: dx[M][K] = dY[M][N] . W[N][K]     dY in 1 x 128 blocks along N, W in 128 x 128
 *   wgrad: dw[N][K] = dY[M][N]^T . X[M][K]   both in 1 x 128 blocks along the tokens M
 * Inputs bf16, dense row-major, 2-byte aligned; out dense row-major of out_dtype. Any sizes
 * 0 <= M, K, N <= 2^23 with fewer than 2^24 tiles of 128 x 128 in the inputs and 2^23 of 256 x 256 in out. ws: at least mxfp4_fp8_linear_workspace_bytes() bytes.
 */
size_t mxfp4_fp8_linear_workspace_bytes(mxfp4_pass_t pass, int64_t M, int64_t K, int64_t N);
mxfp4_status_t mxfp4_fp8_linear_fprop(const void *x_bf16, const void *w_bf16, int64_t M, int64_t K, int64_t N, void *ws,
                                      size_t ws_bytes, void *y, mxfp4_out_dtype_t out_dtype, void *stream);
mxfp4_status_t mxfp4_fp8_linear_dgrad(const void *dy_bf16, const void *w_bf16, int64_t M, int64_t K, int64_t N, void *ws,
                                      size_t ws_bytes, void *dx, mxfp4_out_dtype_t out_dtype, void *stream);
mxfp4_status_t mxfp4_fp8_linear_wgrad(const void *dy_bf16, const void *x_bf16, int64_t M, int64_t K, int64_t N, void *ws,
                                      size_t ws_bytes, void *dw, mxfp4_out_dtype_t out_dtype, void *stream);

/* ---------------------------------------------------------------------------------------------
 * Softmax cross entropy of a linear head.
 *
 *   z = X W^T (bf16 operands, FP32 products, never stored),  lse_t = log sum_v exp z_tv,
 *   loss_t = lse_t - z_t,target(t)   (0 where target(t) == ignore_index; NaN where it is no index)
 *
 * X[T][ldx], W[V][ldw] bf16; target int64 [T]; loss and lse FP32 [T]. With K % 64 == 0 both are read in
 * place and need 16-byte aligned rows (pointer, and ldx, ldw multiples of 8); any other K is copied
 * into the workspace first, padded, and needs no alignment. A row of logits with a NaN or +infinity
 * gives NaN. The caller reduces the losses as it likes: the backward
 * call takes the gradient of each row's loss, and of each row's lse (for a penalty on it).
 *
 *   G_tv = exp(z_tv - lse_t) (dloss_t + dlse_t) - [v = target(t)] dloss_t
 *   dX = G W,  dW = G^T X
 *
 * dloss, dlse FP32 [T], either may be NULL (zeros); a row whose target is ignore_index or no index
 * counts with dloss_t = 0. A row with dloss_t = dlse_t = 0 adds nothing, whatever it holds (NaN in X
 * included). lse is the forward call's. The products of the gradients take FP16 operands, G, X and W each
 * scaled by a power of two to FP16's range: an entry of G is rounded to half a step of FP16 (2^-11 of
 * itself) after the exponential has taken over the roundings of z and of lse (an error d of z - lse is one
 * of d |dloss + dlse| p, at the target too, where p - 1 may be small beside it), and entries of G, X and W below 2^-28 of the largest finite one (of |dloss| + |dloss + dlse|
 * for G) to 2^-39 of that. A NaN or an infinity in one row's gradient or in W has the products it has in
 * the formula, and no say in those scales. dx [T][K] and dw [V][K], dense, FP32 or bf16; either
 * may be NULL, and is then not computed.
 * Requirements: T >= 0, K, V >= 1, below 2^21 (T, K) and 2^31 (V); ldx, ldw >= K and below 2^21; in the
 * backward call fewer than 2^24 tiles of 128 x 128 in X and in a piece of W together.
 * Workspaces: the forward call keeps 8 bytes for each row and each 256 (few rows: 128 or 64) columns; the
 * backward call two copies of G, in FP16 and of 256 MB each or less, but at least 1280 columns (so more
 * from 2^16 tokens on: 8 GB each at 2^21), and X and a piece of W in FP16.
 * T == 0 returns MXFP4_OK after setting dw, if given, to zero.
 */
size_t mxfp4_linear_xent_forward_workspace_bytes(int64_t T, int64_t K, int64_t V);
size_t mxfp4_linear_xent_backward_workspace_bytes(int64_t T, int64_t K, int64_t V);
mxfp4_status_t mxfp4_linear_xent_forward(const void *x_bf16, int64_t ldx, const void *w_bf16, int64_t ldw,
                                         const int64_t *target, int64_t T, int64_t K, int64_t V, int64_t ignore_index,
                                         void *ws, size_t ws_bytes, float *loss, float *lse, void *stream);
mxfp4_status_t mxfp4_linear_xent_backward(const float *dloss, const float *dlse, const void *x_bf16, int64_t ldx,
                                          const void *w_bf16, int64_t ldw, const int64_t *target, const float *lse,
                                          int64_t T, int64_t K, int64_t V, int64_t ignore_index, void *ws, size_t ws_bytes,
                                          void *dx, mxfp4_out_dtype_t dx_dtype, void *dw, mxfp4_out_dtype_t dw_dtype,
                                          void *stream);

/* ---------------------------------------------------------------------------------------------
 * mxfp4_orthogonalize -- Newton-Schulz orthogonalisation of `batch` matrices G[m][n]:
 *
 *   X = G / (|G|_F + eps);  steps times:  A = X X^T,  X <- a X + (b A + c A A) X
 *   out = alpha * X + beta * out
 *
 * (the Gram matrix along the shorter side). g: bf16 or FP32, row stride ldg, matrices batch_stride_g
 * elements apart; out: FP32 or bf16 with ldo and batch_stride_o; out may be read only when beta != 0
 * and must not overlap g. With a side of at most 64 everything is held in FP32; five steps
 * are off by 1e-6 to 1e-4 of the result's norm. Larger matrices' products take FP16 operands and accumulate
 * in FP32, X is carried in 22 bits: five steps are off by 0.0003 to 0.0018. A bf16 result's own rounding is
 * 0.0017.
 * A matrix that holds a NaN or an infinity gives NaN (that matrix only).
 * Coefficients: finite, and such that singular values that start in [0, 1] stay within 4 and |b x + c x x|
 * within 32 for their squares x at every step (MXFP4_ERR_ARG otherwise: FP16 would overflow);
 * (3.4445, -4.7750, 2.0315) with 5 steps stay within 1.3 and 2.9.
 * Requirements: batch, m, n >= 0, at most 65535, 2^20, 2^20, batch * m * n <= 2^31 and fewer than 2^23
 * tiles of 256 x 256 in the batch; 0 <= steps <= 32; ldg, ldo >= n; with batch > 1 the strides at least m
 * rows.
 */
size_t mxfp4_orthogonalize_workspace_bytes(int64_t batch, int64_t m, int64_t n);
mxfp4_status_t mxfp4_orthogonalize(const void *g, mxfp4_dtype_t dtype, int64_t batch, int64_t m, int64_t n, int64_t ldg,
                                   int64_t batch_stride_g, int steps, float a, float b, float c, float eps, float alpha,
                                   float beta, void *out, mxfp4_out_dtype_t out_dtype, int64_t ldo, int64_t batch_stride_o,
                                   void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_TRAIN_H_ */
