/*
 * mxfp4_layer.h -- C ABI of libmxfp4_layer.so: what a training step does between the products of mxfp4.h and
 * mxfp4_train.h, for AMD MI355X (gfx950). Each of these reads and writes memory once where it can.
 *
 *  - RMS norm of a residual stream (mxfp4_rmsnorm_*), with the addition of a branch in front, the result
 *    in 16 or 32 bits and as 8-bit operands of mxfp4_fp8_gemm, and its gradients;
 *  - the gated activation (mxfp4_swiglu_*): silu(gate) * up, with the same 8-bit operands, and its gradients, which
 *    are 8-bit operands as well;
 *  - the norm over all gradients and their clipping (mxfp4_grad_*).
 *
 * Conventions are those of mxfp4.h: device pointers owned by the caller and only used until the enqueued
 * work ends; asynchronous on `stream`; argument errors found before any launch, nothing launched and no output
 * touched; workspaces given by the caller (256-byte aligned, in use until the work ends: two calls, or two captured
 * graphs, that may run at the same time need one each); no state between calls; results that do not change from run
 * to run (no atomics); gfx950 only. Every call can be captured into a graph.
 *
 * Matrices are row-major with a row stride (ld) in elements, at least the columns; pointers need their element's
 * alignment only (rows at multiples of 16 bytes are read faster). A matrix may be NULL where that is said.
 * Outputs overlap nothing unless that is said; two outputs never overlap.
 *
 * 8-bit outputs are those of mxfp4_fp8_quantize with MXFP4_FP8_ROW: E4M3 codes and a power-of-two scale byte for
 * each 128 values, formed of the FP32 value (not of one rounded to bf16 first).
 *   q1, ldq1, s1, lds1   along the rows: outer = rows, L = cols; q1 = NULL: not wanted
 *   q0, ldq0, s0, lds0   along the columns, the quantized transpose: outer = cols, L = rows; or q0 = NULL
 * ldq >= round_up(L, 128) and a multiple of 16, q 16-byte aligned, lds >= ceil(L / 128). Codes behind L are
 * zero. A block that holds a NaN or an infinity has the scale 0xFF and zero codes.
 */
#ifndef MXFP4_LAYER_H_
#define MXFP4_LAYER_H_

#include "mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Raised whenever an entry point, an argument's meaning or a layout changes. */
#define MXFP4_LAYER_ABI_VERSION 1

/* MXFP4_LAYER_ABI_VERSION of the built library. */
int mxfp4_layer_abi_version(void);

/* ---------------------------------------------------------------------------------------------
 * RMS norm.
 *
 *   h = x + residual, rounded to stream_dtype       (h = x without a residual)
 *   rstd_t = 1 / sqrt(mean over k of h_tk^2 + eps)
 *   y_tk = (h_tk * rstd_t) * weight_k               (weight NULL: ones)
 *
 * The squares are summed in 64 bits, rstd is rounded to FP32 and y formed in FP32. A row that holds a NaN
 * gives NaN; one with an infinity 0, and NaN at the infinity; a row of zeros with eps = 0 NaN. Root mean squares
 * below 2^-126 or above 2^126 lose bits in rstd, which FP32 does not hold there.
 *   x         [rows][ldx] of x_dtype
 *   residual  [rows][ldr] of stream_dtype, or NULL; h [rows][ldh] of stream_dtype, its sum with x, or NULL (not
 *             wanted; without a residual it has to be NULL). h may be residual, or x where the types are
 *             the same (with the same row stride).
 *   weight    [cols] of w_dtype, or NULL
 *   rstd      FP32 [rows], or NULL;  y [rows][ldy] of y_dtype, or NULL
 * Codes along the columns are formed in a second pass over h: they need rstd, and with a residual h.
 * Requirements: 0 <= rows < 2^31, 1 <= cols <= 2^24; with q0 fewer than 2^23 tiles of 128 x 128; eps >= 0 and finite.
 *
 *   u_tk = dy_tk weight_k
 *   dh_tk = rstd_t u_tk - h_tk rstd_t^3 mean over j of (u_tj h_tj) + dres_tk     (the gradient of x and of residual)
 *   dweight_k = sum over t of dy_tk h_tk rstd_t
 *
 *   dy [rows][lddy] of dy_dtype;  dres [rows][lddr], the gradient that arrives at h along the stream, h, and dh
 *   [rows][lddh] of stream_dtype; dres may be NULL (zeros), dh may be dres (with the same row stride).
 *   rstd is the forward call's; dweight [cols] of dw_dtype, or NULL (then no workspace is needed). rows == 0 sets it to zero.
 * All of it in FP32; the rows' sum for dweight in a fixed order.
 */
mxfp4_status_t mxfp4_rmsnorm_forward(const void *x, mxfp4_dtype_t x_dtype, int64_t ldx, const void *residual, int64_t ldr,
                                     mxfp4_dtype_t stream_dtype, const void *weight, mxfp4_dtype_t w_dtype, int64_t rows,
                                     int64_t cols, float eps, void *h, int64_t ldh, float *rstd, void *y,
                                     mxfp4_out_dtype_t y_dtype, int64_t ldy, uint8_t *q1, int64_t ldq1, uint8_t *s1,
                                     int64_t lds1, uint8_t *q0, int64_t ldq0, uint8_t *s0, int64_t lds0, void *stream);
size_t mxfp4_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols);
mxfp4_status_t mxfp4_rmsnorm_backward(const void *dy, mxfp4_dtype_t dy_dtype, int64_t lddy, const void *dres, int64_t lddr,
                                      const void *h, int64_t ldh, mxfp4_dtype_t stream_dtype, const void *weight,
                                      mxfp4_dtype_t w_dtype, const float *rstd, int64_t rows, int64_t cols, void *dh,
                                      int64_t lddh, void *dweight, mxfp4_out_dtype_t dw_dtype, void *ws, size_t ws_bytes,
                                      void *stream);

/* ---------------------------------------------------------------------------------------------
 * Gated activation.
 *
 *   s = 1 / (1 + exp(-gate));  a = gate s up
 *   dgate = da up s (1 + gate (1 - s));  dup = da gate s
 *
 *   gate [rows][ldg], up [rows][ldu] of dtype; a [rows][lda] of a_dtype, or NULL; da [rows][ldda] of da_dtype;
 *   dgate [rows][lddg], dup [rows][lddu] of out_dtype, either may be NULL.
 * gate and up may be the halves of one matrix, as a fused product writes it. So may the gradients: with cols a
 * multiple of 128, q1_up = q1_gate + cols and s1_up = s1_gate + cols / 128 make one operand of 2 cols a row, and
 * q0_up = q0_gate + cols * ldq0, s0_up = s0_gate + cols * lds0 one of 2 cols rows (with any cols). q1_gate and q1_up
 * have one ldq1 and lds1, q0_gate and q0_up one ldq0 and lds0.
 * a may be gate or up, and dgate and dup may be any two of gate, up and da, with the same type and row stride.
 * All of it in FP32, the products as (gate s) up, da (gate s) and da (up (s (1 + gate (1 - s)))). Where the results and what stands
 * in brackets are in FP32's normal range, a and dup are off by at most 2^-21 of themselves and dgate by 2^-20 of
 * |da up s| (1 + |gate (1 - s)|), before the rounding to their types (da up alone may overflow); an s or 1 - s below
 * 2^-126 may be lost (gates beyond 87).
 * NaN as in the formulas.
 * Requirements: 0 <= rows, cols < 2^31; fewer than 2^23 tiles of 128 x 128.
 */
mxfp4_status_t mxfp4_swiglu_forward(const void *gate, int64_t ldg, const void *up, int64_t ldu, mxfp4_dtype_t dtype,
                                    int64_t rows, int64_t cols, void *a, mxfp4_out_dtype_t a_dtype, int64_t lda, uint8_t *q1,
                                    int64_t ldq1, uint8_t *s1, int64_t lds1, uint8_t *q0, int64_t ldq0, uint8_t *s0,
                                    int64_t lds0, void *stream);
mxfp4_status_t mxfp4_swiglu_backward(const void *da, mxfp4_dtype_t da_dtype, int64_t ldda, const void *gate, int64_t ldg,
                                     const void *up, int64_t ldu, mxfp4_dtype_t dtype, int64_t rows, int64_t cols, void *dgate,
                                     int64_t lddg, void *dup, int64_t lddu, mxfp4_out_dtype_t out_dtype, uint8_t *q1_gate,
                                     uint8_t *q1_up, int64_t ldq1, uint8_t *s1_gate, uint8_t *s1_up, int64_t lds1,
                                     uint8_t *q0_gate, uint8_t *q0_up, int64_t ldq0, uint8_t *s0_gate, uint8_t *s0_up,
                                     int64_t lds0, void *stream);

/* ---------------------------------------------------------------------------------------------
 * The norm over n tensors of gradients together, and their clipping.
 *
 *   norm = sqrt(sum over all values of g^2)
 *   out = g * min(1, max_norm / (norm + eps))
 *
 * g: `count` values of dtype, dense; out: as many of out_dtype, or g itself (in place, the types being the same).
 * Squares are summed in 64 bits, so FP32 values of any size count; norm is rounded to FP32 at the end. An infinite
 * norm makes finite values 0 and infinities NaN, one that is NaN everything NaN, as the formula has it.
 * In place with norm + eps <= max_norm nothing is written.
 *
 * mxfp4_grad_clip does both. The other two are its halves, for gradients that are spread over several cards: the
 * ranks add up sum_sq (one 64-bit value on the device) between them.
 *   sum_sq  [1] on the device, the sum of the squares: written by grad_norm (or NULL), read by grad_scale
 *   norm    FP32 [1] on the device, or NULL
 * The arrays of mxfp4_grad_t are host memory and only read during the call; tensors go to the device in the
 * kernels' arguments, 224 a launch for the sums and 160 for the scaling.
 * Requirements: 0 <= n < 2^20; 0 <= count <= 2^37; max_norm > 0 and finite, eps >= 0 and finite. In mxfp4_grad_scale and
 * mxfp4_grad_clip no out may overlap another out or another tensor's g (MXFP4_ERR_ARG). ws: at least
 * mxfp4_grad_norm_workspace_bytes() bytes.
 */
typedef struct {
    const void *g;
    void *out;                      /* not used by mxfp4_grad_norm */
    int64_t count;
    mxfp4_dtype_t dtype;
    mxfp4_out_dtype_t out_dtype;
} mxfp4_grad_t;
size_t mxfp4_grad_norm_workspace_bytes(const mxfp4_grad_t *grads, int64_t n);
mxfp4_status_t mxfp4_grad_norm(const mxfp4_grad_t *grads, int64_t n, void *ws, size_t ws_bytes, double *sum_sq, float *norm,
                               void *stream);
mxfp4_status_t mxfp4_grad_scale(const mxfp4_grad_t *grads, int64_t n, const double *sum_sq, float max_norm, float eps,
                                float *norm, void *stream);
mxfp4_status_t mxfp4_grad_clip(const mxfp4_grad_t *grads, int64_t n, float max_norm, float eps, void *ws, size_t ws_bytes,
                               float *norm, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_LAYER_H_ */
