// C-ABI entry points of libmxfp4_train: argument validation, workspace carve-up and dispatch.
// Every argument check happens before the first HIP call, so an invalid call launches nothing,
// touches no output and needs no device.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/mxfp4_train.h"
#include "train_internal.h"

namespace {

constexpr int64_t kMaxDim = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxLinear = (int64_t)1 << 23;

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

mxfp4_status_t check_device()
{
    // gfx950 check, cached per device ordinal: 0 = unknown, 1 = gfx950, 2 = other
    static std::atomic<int> cache[64];
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return MXFP4_ERR_DEVICE;
    if (dev < 64) {
        const int known = cache[dev].load(std::memory_order_relaxed);
        if (known) return known == 1 ? MXFP4_OK : MXFP4_ERR_DEVICE;
    }
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MXFP4_ERR_DEVICE;
    const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev < 64) cache[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
    return ok ? MXFP4_OK : MXFP4_ERR_DEVICE;
}

mxfp4_status_t from_hip(hipError_t e) { return e == hipSuccess ? MXFP4_OK : MXFP4_ERR_LAUNCH; }

bool valid_out(int t) { return t == MXFP4_OUT_F32 || t == MXFP4_OUT_BF16; }
size_t out_size(int t) { return t == MXFP4_OUT_BF16 ? 2 : 4; }
bool in_range(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

int64_t fp8_tiles(int64_t rows, int64_t cols) { return (rows + 127) / 128 * ((cols + 127) / 128); }

mxfp4_status_t check_fp8_out(const uint8_t *q, int64_t ldq, const uint8_t *s, int64_t lds, int64_t L)
{
    if (ldq < mx::round_up(L, 128) || lds < (L + 127) / 128 || lds < 1) return MXFP4_ERR_ARG;
    if (!s) return MXFP4_ERR_NULL;
    if (!aligned(q, 16) || ldq % 16 != 0) return MXFP4_ERR_ALIGN;
    return MXFP4_OK;
}

// Quantized operand of a linear call in the workspace.
struct Operand {
    int64_t outer, L;
    int64_t ldq() const { return mx::round_up(L, 128); }
    int64_t lds() const { return mx::round_up((L + 127) / 128, 16); }
    size_t codes() const { return (size_t)mx::round_up(outer * ldq(), 256); }
    size_t scales() const { return (size_t)mx::round_up(outer * lds(), 256); }
    size_t bytes() const { return codes() + scales(); }
    mx::Fp8Out at(uint8_t *p) const { return mx::Fp8Out{p, ldq(), p + codes(), lds()}; }
};
struct LinearPlan {
    Operand a, b;   // the product is a.outer x b.outer over a.L = b.L
};
bool linear_plan(int pass, int64_t M, int64_t K, int64_t N, LinearPlan &p)
{
    if (!in_range(M, 0, kMaxLinear) || !in_range(K, 0, kMaxLinear) || !in_range(N, 0, kMaxLinear)) return false;
    switch (pass) {
    case MXFP4_FPROP: p = {{M, K}, {N, K}}; break;
    case MXFP4_DGRAD: p = {{M, N}, {K, N}}; break;
    case MXFP4_WGRAD: p = {{N, M}, {K, M}}; break;
    default: return false;
    }
    // what the two launches can hold
    return fp8_tiles(p.a.outer, p.a.L) + fp8_tiles(p.b.outer, p.b.L) <= mx::kFp8Tiles &&
           mx::product_fits_grid(p.a.outer, p.b.outer);
}
size_t linear_bytes(const LinearPlan &p)
{
    return p.a.bytes() + p.b.bytes() + mx::fp8_gemm_workspace_bytes(p.a.outer, p.b.outer, p.a.L);
}

mxfp4_status_t run_linear(int pass, const void *a, const void *b, int64_t M, int64_t K, int64_t N, void *ws,
                          size_t ws_bytes, void *out, int out_dtype, void *stream)
{
    LinearPlan p;
    if (!linear_plan(pass, M, K, N, p)) return MXFP4_ERR_SHAPE;
    if (!valid_out(out_dtype)) return MXFP4_ERR_ARG;
    if (p.a.outer == 0 || p.b.outer == 0) return MXFP4_OK;
    if (!out || (p.a.L > 0 && (!a || !b || !ws))) return MXFP4_ERR_NULL;
    if (!aligned(a, 2) || !aligned(b, 2) || !aligned(out, out_size(out_dtype)) || !aligned(ws, 256)) return MXFP4_ERR_ALIGN;
    if (p.a.L > 0 && ws_bytes < linear_bytes(p)) return MXFP4_ERR_WORKSPACE;
    const mxfp4_status_t dev = check_device();
    if (dev != MXFP4_OK) return dev;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool bf16 = out_dtype == MXFP4_OUT_BF16;
    if (p.a.L == 0) return from_hip(mx::launch_scale_output(out, bf16, p.a.outer, p.b.outer, p.b.outer, 0.0f, s));
    uint8_t *w = static_cast<uint8_t *>(ws);
    const mx::Fp8Out qa = p.a.at(w), qb = p.b.at(w + p.a.bytes()), none{};
    // rows x cols of the two inputs as they lie in memory, and which axis is quantized
    const bool tile = pass != MXFP4_WGRAD;
    mx::Fp8Input in[2];
    const bool a1 = pass != MXFP4_WGRAD, b1 = pass == MXFP4_FPROP;
    in[0] = {a, M, pass == MXFP4_FPROP ? K : N, pass == MXFP4_FPROP ? K : N, false, false, a1 ? qa : none, a1 ? none : qa};
    in[1] = {b, pass == MXFP4_WGRAD ? M : N, K, K, false, tile, b1 ? qb : none, b1 ? none : qb};
    if (hipError_t e = mx::launch_fp8_quantize(in, 2, s)) return from_hip(e);
    uint8_t *split = w + p.a.bytes() + p.b.bytes();
    return from_hip(mx::launch_fp8_gemm(qa.q, qa.ldq, qa.s, qa.lds, qb.q, qb.ldq, qb.s, qb.lds, p.a.outer, p.b.outer, p.a.L,
                                        1.0f, 0.0f, out, bf16, p.b.outer, split,
                                        mx::fp8_gemm_workspace_bytes(p.a.outer, p.b.outer, p.a.L), s));
}

// -------------------------------------------------------------------------------- head loss ---
constexpr int64_t kMaxTokens = ((int64_t)1 << 21) - 1;

bool xent_sizes(int64_t T, int64_t K, int64_t V)
{
    return in_range(T, 0, kMaxTokens) && in_range(K, 1, kMaxTokens) && in_range(V, 1, kMaxDim);
}
mxfp4_status_t check_xent(const void *x, int64_t ldx, const void *w, int64_t ldw, const int64_t *target, int64_t T,
                          int64_t K, int64_t V)
{
    if (!xent_sizes(T, K, V)) return MXFP4_ERR_SHAPE;
    if (!in_range(ldx, K, kMaxTokens) || !in_range(ldw, K, kMaxTokens)) return MXFP4_ERR_ARG;
    if (T == 0) return MXFP4_OK;
    if (!x || !w || !target) return MXFP4_ERR_NULL;
    if (!aligned(x, 2) || !aligned(w, 2) || !aligned(target, 8)) return MXFP4_ERR_ALIGN;
    if (K % 64 == 0 && (!aligned(x, 16) || !aligned(w, 16) || ldx % 8 != 0 || ldw % 8 != 0)) return MXFP4_ERR_ALIGN;
    return MXFP4_OK;
}

// --------------------------------------------------------------------------- Newton-Schulz ----
bool ortho_sizes(int64_t batch, int64_t m, int64_t n)
{
    const int64_t most = (int64_t)1 << 20;
    if (!in_range(batch, 0, 65535) || !in_range(m, 0, most) || !in_range(n, 0, most)) return false;
    if (batch == 0 || m == 0 || n == 0) return true;
    return n <= ((int64_t)1 << 31) / batch / m && mx::product_fits_grid(m, n, batch);
}
// The scalar iteration against the range that FP16 holds. The values reached from [0, 1] are, up to their sign, an interval
// [0, top] at every step (the step is continuous, odd, and 0 at 0), whose next end is the largest |step| at its end or where
// the slope a + 3 b x + 5 c x x, x the square, vanishes. (A grid of starting values misses narrow ranges of them that
// leave it after several steps.)
bool ortho_bounded(int steps, float af, float bf, float cf)
{
    if (!std::isfinite(af) || !std::isfinite(bf) || !std::isfinite(cf)) return false;
    const double a = af, b = bf, c = cf;
    const auto poly = [&](double x) { return b * x + c * x * x; };
    // places of extrema; those that do not exist come out as NaN or outside every interval
    const double vertex = -b / (2.0 * c), root = -1.5 * b - std::copysign(0.5 * std::sqrt(9.0 * b * b - 20.0 * a * c), b);
    const double flat[2] = {root / (5.0 * c), a / root};
    double top = 1.0;
    for (int k = 0; k < steps; ++k) {
        const double end = top * top;
        double high = std::fabs(poly(end));
        if (vertex > 0.0 && vertex < end) high = std::max(high, std::fabs(poly(vertex)));
        if (high > 32.0) return false;
        top = std::fabs((a + poly(end)) * top);
        for (const double x : flat)
            if (x > 0.0 && x < end) top = std::max(top, std::fabs((a + poly(x)) * std::sqrt(x)));
        if (top > 4.0) return false;
    }
    return true;
}

}  // namespace

extern "C" {

int mxfp4_train_abi_version(void) { return MXFP4_TRAIN_ABI_VERSION; }

mxfp4_status_t mxfp4_fp8_quantize(const void *x, mxfp4_dtype_t dtype, int64_t rows, int64_t cols, int64_t ldx,
                                  mxfp4_fp8_block_t block, uint8_t *q1, int64_t ldq1, uint8_t *s1, int64_t lds1,
                                  uint8_t *q0, int64_t ldq0, uint8_t *s0, int64_t lds0, void *stream)
{
    if (dtype != MXFP4_IN_BF16 && dtype != MXFP4_IN_F32) return MXFP4_ERR_ARG;
    if (block != MXFP4_FP8_ROW && block != MXFP4_FP8_TILE) return MXFP4_ERR_ARG;
    if (!in_range(rows, 0, kMaxDim) || !in_range(cols, 0, kMaxDim)) return MXFP4_ERR_SHAPE;
    if (fp8_tiles(rows, cols) > mx::kFp8Tiles) return MXFP4_ERR_SHAPE;
    if (ldx < cols || ldx < 1) return MXFP4_ERR_ARG;
    if (rows == 0 || cols == 0) return MXFP4_OK;
    if (!x || (!q1 && !q0)) return MXFP4_ERR_NULL;
    if (q1)
        if (mxfp4_status_t e = check_fp8_out(q1, ldq1, s1, lds1, cols)) return e;
    if (q0)
        if (mxfp4_status_t e = check_fp8_out(q0, ldq0, s0, lds0, rows)) return e;
    if (!aligned(x, dtype == MXFP4_IN_F32 ? 4 : 2)) return MXFP4_ERR_ALIGN;
    const mxfp4_status_t dev = check_device();
    if (dev != MXFP4_OK) return dev;
    const mx::Fp8Input in{x, rows, cols, ldx, dtype == MXFP4_IN_F32, block == MXFP4_FP8_TILE, {q1, ldq1, s1, lds1},
                          {q0, ldq0, s0, lds0}};
    return from_hip(mx::launch_fp8_quantize(&in, 1, static_cast<hipStream_t>(stream)));
}

size_t mxfp4_fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (!in_range(M, 1, kMaxDim) || !in_range(N, 1, kMaxDim) || !in_range(K, 1, kMaxDim) || !mx::product_fits_grid(M, N)) return 0;
    return mx::fp8_gemm_workspace_bytes(M, N, K);
}

mxfp4_status_t mxfp4_fp8_gemm(const uint8_t *aq, int64_t lda, const uint8_t *as, int64_t ldas, const uint8_t *bq,
                              int64_t ldb, const uint8_t *bs, int64_t ldbs, int64_t M, int64_t N, int64_t K, float alpha,
                              float beta, void *c, mxfp4_out_dtype_t c_dtype, int64_t ldc, void *workspace, size_t ws_bytes,
                              void *stream)
{
    if (!valid_out(c_dtype)) return MXFP4_ERR_ARG;
    if (!in_range(M, 0, kMaxDim) || !in_range(N, 0, kMaxDim) || !in_range(K, 0, kMaxDim)) return MXFP4_ERR_SHAPE;
    const int64_t kp = mx::round_up(K, 128), kb = (K + 127) / 128, most = ((int64_t)1 << 24) - 1;
    if (ldc < N || ldc < 1) return MXFP4_ERR_ARG;
    if (!in_range(lda, kp, most) || !in_range(ldb, kp, most) || !in_range(ldas, kb, most) || !in_range(ldbs, kb, most))
        return MXFP4_ERR_ARG;
    if (M == 0 || N == 0) return MXFP4_OK;
    if (!mx::product_fits_grid(M, N)) return MXFP4_ERR_SHAPE;
    if (!c || (K > 0 && (!aq || !as || !bq || !bs))) return MXFP4_ERR_NULL;
    if (!aligned(c, out_size(c_dtype))) return MXFP4_ERR_ALIGN;
    if (K > 0 && (!aligned(aq, 16) || !aligned(bq, 16) || !aligned(as, 16) || !aligned(bs, 16) || lda % 16 || ldb % 16 ||
                  ldas % 16 || ldbs % 16))
        return MXFP4_ERR_ALIGN;
    if (workspace && !aligned(workspace, 256)) return MXFP4_ERR_ALIGN;
    const mxfp4_status_t dev = check_device();
    if (dev != MXFP4_OK) return dev;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool bf16 = c_dtype == MXFP4_OUT_BF16;
    if (K == 0) return from_hip(mx::launch_scale_output(c, bf16, M, N, ldc, beta, s));
    return from_hip(mx::launch_fp8_gemm(aq, lda, as, ldas, bq, ldb, bs, ldbs, M, N, K, alpha, beta, c, bf16, ldc, workspace,
                                        workspace ? ws_bytes : 0, s));
}

size_t mxfp4_fp8_linear_workspace_bytes(mxfp4_pass_t pass, int64_t M, int64_t K, int64_t N)
{
    LinearPlan p;
    return linear_plan(pass, M, K, N, p) ? linear_bytes(p) : 0;
}
mxfp4_status_t mxfp4_fp8_linear_fprop(const void *x, const void *w, int64_t M, int64_t K, int64_t N, void *ws, size_t ws_bytes,
                                      void *y, mxfp4_out_dtype_t out_dtype, void *stream)
{
    return run_linear(MXFP4_FPROP, x, w, M, K, N, ws, ws_bytes, y, out_dtype, stream);
}
mxfp4_status_t mxfp4_fp8_linear_dgrad(const void *dy, const void *w, int64_t M, int64_t K, int64_t N, void *ws, size_t ws_bytes,
                                      void *dx, mxfp4_out_dtype_t out_dtype, void *stream)
{
    return run_linear(MXFP4_DGRAD, dy, w, M, K, N, ws, ws_bytes, dx, out_dtype, stream);
}
mxfp4_status_t mxfp4_fp8_linear_wgrad(const void *dy, const void *x, int64_t M, int64_t K, int64_t N, void *ws, size_t ws_bytes,
                                      void *dw, mxfp4_out_dtype_t out_dtype, void *stream)
{
    return run_linear(MXFP4_WGRAD, dy, x, M, K, N, ws, ws_bytes, dw, out_dtype, stream);
}

size_t mxfp4_linear_xent_forward_workspace_bytes(int64_t T, int64_t K, int64_t V)
{
    return T > 0 && xent_sizes(T, K, V) ? mx::xent_forward_workspace_bytes(T, K, V) : 0;
}
size_t mxfp4_linear_xent_backward_workspace_bytes(int64_t T, int64_t K, int64_t V)
{
    return T > 0 && xent_sizes(T, K, V) && mx::xent_backward_fits_grid(T, K, V) ? mx::xent_backward_workspace_bytes(T, K, V) : 0;
}

mxfp4_status_t mxfp4_linear_xent_forward(const void *x, int64_t ldx, const void *w, int64_t ldw, const int64_t *target,
                                         int64_t T, int64_t K, int64_t V, int64_t ignore_index, void *ws, size_t ws_bytes,
                                         float *loss, float *lse, void *stream)
{
    if (mxfp4_status_t e = check_xent(x, ldx, w, ldw, target, T, K, V)) return e;
    if (T == 0) return MXFP4_OK;
    if (!loss || !lse || !ws) return MXFP4_ERR_NULL;
    if (!aligned(loss, 4) || !aligned(lse, 4) || !aligned(ws, 256)) return MXFP4_ERR_ALIGN;
    if (ws_bytes < mx::xent_forward_workspace_bytes(T, K, V)) return MXFP4_ERR_WORKSPACE;
    const mxfp4_status_t dev = check_device();
    if (dev != MXFP4_OK) return dev;
    const mx::XentProblem p{x, w, ldx, ldw, target, T, K, V, ignore_index};
    return from_hip(mx::launch_xent_forward(p, ws, loss, lse, static_cast<hipStream_t>(stream)));
}

mxfp4_status_t mxfp4_linear_xent_backward(const float *dloss, const float *dlse, const void *x, int64_t ldx, const void *w,
                                          int64_t ldw, const int64_t *target, const float *lse, int64_t T, int64_t K,
                                          int64_t V, int64_t ignore_index, void *ws, size_t ws_bytes, void *dx,
                                          mxfp4_out_dtype_t dx_dtype, void *dw, mxfp4_out_dtype_t dw_dtype, void *stream)
{
    if ((dx && !valid_out(dx_dtype)) || (dw && !valid_out(dw_dtype))) return MXFP4_ERR_ARG;
    if (mxfp4_status_t e = check_xent(x, ldx, w, ldw, target, T, K, V)) return e;
    if (T > 0 && !mx::xent_backward_fits_grid(T, K, V)) return MXFP4_ERR_SHAPE;
    if (!dx && !dw) return MXFP4_OK;
    if ((dx && !aligned(dx, out_size(dx_dtype))) || (dw && !aligned(dw, out_size(dw_dtype)))) return MXFP4_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T > 0) {
        if (!lse || !ws) return MXFP4_ERR_NULL;
        if (!aligned(dloss, 4) || !aligned(dlse, 4) || !aligned(lse, 4) || !aligned(ws, 256)) return MXFP4_ERR_ALIGN;
        if (ws_bytes < mx::xent_backward_workspace_bytes(T, K, V)) return MXFP4_ERR_WORKSPACE;
    }
    if (T == 0 && !dw) return MXFP4_OK;
    const mxfp4_status_t dev = check_device();
    if (dev != MXFP4_OK) return dev;
    if (T == 0) return from_hip(mx::launch_scale_output(dw, dw_dtype == MXFP4_OUT_BF16, V, K, K, 0.0f, s));
    const mx::XentProblem p{x, w, ldx, ldw, target, T, K, V, ignore_index};
    return from_hip(mx::launch_xent_backward(p, dloss, dlse, lse, ws, dx, dx_dtype == MXFP4_OUT_BF16, dw,
                                             dw_dtype == MXFP4_OUT_BF16, s));
}

size_t mxfp4_orthogonalize_workspace_bytes(int64_t batch, int64_t m, int64_t n)
{
    return ortho_sizes(batch, m, n) && batch && m && n ? mx::ortho_workspace_bytes(batch, m, n) : 0;
}

mxfp4_status_t mxfp4_orthogonalize(const void *g, mxfp4_dtype_t dtype, int64_t batch, int64_t m, int64_t n, int64_t ldg,
                                   int64_t batch_stride_g, int steps, float a, float b, float c, float eps, float alpha,
                                   float beta, void *out, mxfp4_out_dtype_t out_dtype, int64_t ldo, int64_t batch_stride_o,
                                   void *ws, size_t ws_bytes, void *stream)
{
    if (dtype != MXFP4_IN_BF16 && dtype != MXFP4_IN_F32) return MXFP4_ERR_ARG;
    if (!valid_out(out_dtype)) return MXFP4_ERR_ARG;
    if (!ortho_sizes(batch, m, n)) return MXFP4_ERR_SHAPE;
    if (!in_range(steps, 0, 32) || !ortho_bounded(steps, a, b, c)) return MXFP4_ERR_ARG;
    if (!(eps >= 0.0f)) return MXFP4_ERR_ARG;
    if (ldg < n || ldo < n || ldg < 1 || ldo < 1) return MXFP4_ERR_ARG;
    if (m > 0 && (ldg > INT64_MAX / 4 / m || ldo > INT64_MAX / 4 / m)) return MXFP4_ERR_ARG;
    if (batch > 1 && (batch_stride_g < (m - 1) * ldg + n || batch_stride_o < (m - 1) * ldo + n)) return MXFP4_ERR_ARG;
    if (batch == 0 || m == 0 || n == 0) return MXFP4_OK;
    if (!g || !out || !ws) return MXFP4_ERR_NULL;
    if (!aligned(g, dtype == MXFP4_IN_F32 ? 4 : 2) || !aligned(out, out_size(out_dtype)) || !aligned(ws, 256))
        return MXFP4_ERR_ALIGN;
    if (ws_bytes < mx::ortho_workspace_bytes(batch, m, n)) return MXFP4_ERR_WORKSPACE;
    const mxfp4_status_t dev = check_device();
    if (dev != MXFP4_OK) return dev;
    const mx::OrthoProblem p{g, dtype == MXFP4_IN_F32, batch, m, n, ldg, batch_stride_g, steps, a, b, c, eps, alpha, beta, out,
                             out_dtype == MXFP4_OUT_BF16, ldo, batch_stride_o};
    return from_hip(mx::launch_ortho(p, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
