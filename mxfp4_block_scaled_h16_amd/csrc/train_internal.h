// Launchers behind libmxfp4_train's C ABI (not part of the public interface). Arguments are
// validated by the caller; these pick a kernel and enqueue it.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mx {

// A grid holds fewer than 2^32 work-items along an axis. A product always has a plan when its tiles of 256 x 256, of 512
// threads each, fit one.
constexpr int64_t kMaxItems = ((int64_t)1 << 32) - 1;
constexpr bool product_fits_grid(int64_t M, int64_t N, int64_t batch = 1)
{
    return (M + 255) / 256 * ((N + 255) / 256) * batch <= kMaxItems / 512;
}

constexpr int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// ------------------------------------------------------------------------------- E4M3 ---------
// One operand of an 8-bit product: codes q[outer][ldq] (the first round_up(L, 128) bytes of a row are
// written, zero codes behind L) and E8M0 scales s[outer][lds] (the first ceil(L / 128)).
struct Fp8Out {
    uint8_t *q;
    int64_t ldq;
    uint8_t *s;
    int64_t lds;
};
// x[rows][cols] quantized along its rows (axis1.q != nullptr) and / or its columns (axis0.q != nullptr:
// the quantized transpose), in blocks of 1 x 128 or (tile) 128 x 128.
struct Fp8Input {
    const void *x;
    int64_t rows, cols, ldx;
    bool f32, tile;
    Fp8Out axis1, axis0;
};
constexpr int kFp8Group = 2;
// up to kFp8Group tensors of one type in one launch, of at most kFp8Tiles tiles of 128 x 128 together (256
// threads each)
constexpr int64_t kFp8Tiles = kMaxItems / 256;
hipError_t launch_fp8_quantize(const Fp8Input *items, int count, hipStream_t stream);

// c = alpha A B^T + beta c, FP32 or bf16. K is the row length the scales cover; rows hold
// round_up(K, 128) bytes. workspace: fp8_gemm_workspace_bytes() lets products of few tiles split K.
hipError_t launch_fp8_gemm(const uint8_t *aq, int64_t lda, const uint8_t *as, int64_t ldas, const uint8_t *bq,
                           int64_t ldb, const uint8_t *bs, int64_t ldbs, int64_t M, int64_t N, int64_t K, float alpha,
                           float beta, void *c, bool bf16, int64_t ldc, void *workspace, size_t ws_bytes,
                           hipStream_t stream);
size_t fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);

// c = beta * c (zeros when beta == 0, c not read): the product over an empty contraction
hipError_t launch_scale_output(void *c, bool bf16, int64_t M, int64_t N, int64_t ldc, float beta, hipStream_t stream);

// ------------------------------------------------------------------------------- head loss ----
struct XentProblem {
    const void *x, *w;        // bf16 [T][ldx], [V][ldw]
    int64_t ldx, ldw;
    const int64_t *target;    // [T]
    int64_t T, K, V, ignore_index;
};
size_t xent_forward_workspace_bytes(int64_t T, int64_t K, int64_t V);
size_t xent_backward_workspace_bytes(int64_t T, int64_t K, int64_t V);
bool xent_backward_fits_grid(int64_t T, int64_t K, int64_t V);
hipError_t launch_xent_forward(const XentProblem &p, void *ws, float *loss, float *lse, hipStream_t stream);
// dloss, dlse: [T] or NULL (zeros); dx, dw: NULL or the gradients [T][K], [V][K], FP32 or bf16
hipError_t launch_xent_backward(const XentProblem &p, const float *dloss, const float *dlse, const float *lse, void *ws,
                                void *dx, bool dx_bf16, void *dw, bool dw_bf16, hipStream_t stream);

// --------------------------------------------------------------------------- Newton-Schulz ----
struct OrthoProblem {
    const void *g;
    bool f32;
    int64_t batch, m, n, ldg, batch_g;   // strides in elements
    int steps;
    float a, b, c, eps, alpha, beta;
    void *out;
    bool out_bf16;
    int64_t ldo, batch_o;
};
size_t ortho_workspace_bytes(int64_t batch, int64_t m, int64_t n);
hipError_t launch_ortho(const OrthoProblem &p, void *ws, hipStream_t stream);

}  // namespace mx
