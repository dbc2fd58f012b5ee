// C-ABI entry points of libmxfp4_layer: argument validation and dispatch. Every argument check
// happens before the first HIP call, so an invalid call launches nothing, touches no output and needs no device.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <utility>
#include <vector>

#include "../../include/mxfp4_layer.h"
#include "host_checks.h"
#include "layer_internal.h"

namespace {

using namespace mx;

constexpr int64_t kMaxDim = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxCols = (int64_t)1 << 24;       // a norm's row

int64_t tiles(int64_t rows, int64_t cols) { return (rows + 127) / 128 * ((cols + 127) / 128); }
// a row stride whose offsets in bytes stay in 64 bits
bool stride_ok(int64_t ld, int64_t rows, int64_t cols)
{
    return in_range(ld, std::max<int64_t>(cols, 1), INT64_MAX / 8 / std::max<int64_t>(rows, 1));
}
bool small_finite(float v) { return v >= 0.0f && std::isfinite(v); }

mxfp4_status_t check_both(const Fp8Out &q1, const Fp8Out &q0, int64_t rows, int64_t cols)
{
    if (q1.q)
        if (mxfp4_status_t e = check_fp8_out(q1.q, q1.ldq, q1.s, q1.lds, cols)) return e;
    if (q0.q)
        if (mxfp4_status_t e = check_fp8_out(q0.q, q0.ldq, q0.s, q0.lds, rows)) return e;
    const auto bad = [](const Fp8Out &q, int64_t outer) { return q.q && (!stride_ok(q.ldq, outer, 1) || !stride_ok(q.lds, outer, 1)); };
    return bad(q1, rows) || bad(q0, cols) ? MXFP4_ERR_ARG : MXFP4_OK;
}

// ------------------------------------------------------------------------- gradients' norm ----
constexpr int64_t kMaxGrads = ((int64_t)1 << 20) - 1, kMaxCount = (int64_t)1 << 37;

// Checks the tensors and lists those that hold values. write: their outputs are checked too.
mxfp4_status_t list_grads(const mxfp4_grad_t *grads, int64_t n, bool write, std::vector<GradItem> &items)
{
    if (!in_range(n, 0, kMaxGrads)) return MXFP4_ERR_SHAPE;
    if (n > 0 && !grads) return MXFP4_ERR_NULL;
    items.reserve((size_t)n);
    for (int64_t i = 0; i < n; ++i) {
        const mxfp4_grad_t &t = grads[i];
        if (!valid_in(t.dtype) || (write && !valid_out(t.out_dtype))) return MXFP4_ERR_ARG;
        if (!in_range(t.count, 0, kMaxCount)) return MXFP4_ERR_SHAPE;
        if (t.count == 0) continue;
        if (!t.g || (write && !t.out)) return MXFP4_ERR_NULL;
        if (!aligned(t.g, in_size(t.dtype)) || (write && !aligned(t.out, out_size(t.out_dtype)))) return MXFP4_ERR_ALIGN;
        items.push_back({t.g, t.out, t.count, t.dtype == MXFP4_IN_F32, write && t.out_dtype == MXFP4_OUT_F32});
    }
    if (!write) return MXFP4_OK;
    // a tensor in place is one range; else its g is one that is read and its out one that is written
    struct Range {
        uintptr_t from, to;
        bool written;
        bool operator<(const Range &o) const { return from < o.from; }
    };
    std::vector<Range> ranges;
    ranges.reserve(2 * items.size());
    for (const GradItem &t : items) {
        const uintptr_t g = (uintptr_t)t.g, out = (uintptr_t)t.out;
        const bool in_place = g == out && t.f32 == t.out_f32;
        if (!in_place) ranges.push_back({g, g + (size_t)t.count * (t.f32 ? 4 : 2), false});
        ranges.push_back({out, out + (size_t)t.count * (t.out_f32 ? 4 : 2), true});
    }
    if (!std::is_sorted(ranges.begin(), ranges.end())) std::sort(ranges.begin(), ranges.end());
    // ends of what is written and of what is read so far
    uintptr_t written = 0, read = 0;
    for (const Range &r : ranges) {
        if (r.from < written || (r.written && r.from < read)) return MXFP4_ERR_ARG;
        (r.written ? written : read) = std::max(r.written ? written : read, r.to);
    }
    return MXFP4_OK;
}

// No exception leaves a C entry: a list that finds no memory is a workspace error
template <class F>
mxfp4_status_t guarded(F f)
{
    try {
        return f();
    } catch (...) {
        return MXFP4_ERR_WORKSPACE;
    }
}

}  // namespace

extern "C" {

int mxfp4_layer_abi_version(void) { return MXFP4_LAYER_ABI_VERSION; }

mxfp4_status_t mxfp4_rmsnorm_forward(const void *x, mxfp4_dtype_t x_dtype, int64_t ldx, const void *residual, int64_t ldr,
                                     mxfp4_dtype_t stream_dtype, const void *weight, mxfp4_dtype_t w_dtype, int64_t rows,
                                     int64_t cols, float eps, void *h, int64_t ldh, float *rstd, void *y,
                                     mxfp4_out_dtype_t y_dtype, int64_t ldy, uint8_t *q1, int64_t ldq1, uint8_t *s1,
                                     int64_t lds1, uint8_t *q0, int64_t ldq0, uint8_t *s0, int64_t lds0, void *stream)
{
    if (!valid_in(x_dtype) || (residual && !valid_in(stream_dtype)) || (weight && !valid_in(w_dtype)) ||
        (y && !valid_out(y_dtype)))
        return MXFP4_ERR_ARG;
    if (!in_range(rows, 0, kMaxDim) || !in_range(cols, 1, kMaxCols)) return MXFP4_ERR_SHAPE;
    if (q0 && tiles(rows, cols) > kLayerTiles) return MXFP4_ERR_SHAPE;
    if (!small_finite(eps)) return MXFP4_ERR_ARG;
    if (!stride_ok(ldx, rows, cols) || (residual && !stride_ok(ldr, rows, cols)) || (h && !stride_ok(ldh, rows, cols)) ||
        (y && !stride_ok(ldy, rows, cols)))
        return MXFP4_ERR_ARG;
    if (h && !residual) return MXFP4_ERR_ARG;
    if (rows == 0) return MXFP4_OK;
    if (!x || (q0 && (!rstd || (residual && !h)))) return MXFP4_ERR_NULL;
    const Fp8Out out1{q1, ldq1, s1, lds1}, out0{q0, ldq0, s0, lds0};
    if (mxfp4_status_t e = check_both(out1, out0, rows, cols)) return e;
    if (!aligned(x, in_size(x_dtype)) || (residual && !aligned(residual, in_size(stream_dtype))) ||
        (weight && !aligned(weight, in_size(w_dtype))) || (h && !aligned(h, in_size(stream_dtype))) || !aligned(rstd, 4) ||
        (y && !aligned(y, out_size(y_dtype))))
        return MXFP4_ERR_ALIGN;
    // in place the rows have to be the same ones
    if (h && ((h == residual && ldh != ldr) || (h == x && (ldh != ldx || x_dtype != stream_dtype)))) return MXFP4_ERR_ARG;
    if (!h && !rstd && !y && !q1) return MXFP4_OK;
    const mxfp4_status_t dev = check_device();
    if (dev != MXFP4_OK) return dev;
    const NormForward p{{x, ldx}, {residual, ldr}, weight, x_dtype == MXFP4_IN_F32, stream_dtype == MXFP4_IN_F32,
                        w_dtype == MXFP4_IN_F32, y_dtype == MXFP4_OUT_F32, rows, cols, eps, {h, ldh}, {y, ldy}, rstd, out1, out0};
    return from_hip(launch_norm_forward(p, static_cast<hipStream_t>(stream)));
}

size_t mxfp4_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols)
{
    return in_range(rows, 1, kMaxDim) && in_range(cols, 1, kMaxCols) ? norm_backward_workspace_bytes(rows, cols) : 0;
}

mxfp4_status_t mxfp4_rmsnorm_backward(const void *dy, mxfp4_dtype_t dy_dtype, int64_t lddy, const void *dres, int64_t lddr,
                                      const void *h, int64_t ldh, mxfp4_dtype_t stream_dtype, const void *weight,
                                      mxfp4_dtype_t w_dtype, const float *rstd, int64_t rows, int64_t cols, void *dh,
                                      int64_t lddh, void *dweight, mxfp4_out_dtype_t dw_dtype, void *ws, size_t ws_bytes,
                                      void *stream)
{
    if (!valid_in(dy_dtype) || !valid_in(stream_dtype) || (weight && !valid_in(w_dtype)) || (dweight && !valid_out(dw_dtype)))
        return MXFP4_ERR_ARG;
    if (!in_range(rows, 0, kMaxDim) || !in_range(cols, 1, kMaxCols)) return MXFP4_ERR_SHAPE;
    if (!stride_ok(lddy, rows, cols) || (dres && !stride_ok(lddr, rows, cols)) || !stride_ok(ldh, rows, cols) || !stride_ok(lddh, rows, cols))
        return MXFP4_ERR_ARG;
    if (rows == 0 && !dweight) return MXFP4_OK;
    if (rows > 0 && (!dy || !h || !rstd || !dh || (dweight && !ws))) return MXFP4_ERR_NULL;
    if (dweight && !aligned(dweight, out_size(dw_dtype))) return MXFP4_ERR_ALIGN;
    if (rows > 0) {
        const size_t s = in_size(stream_dtype);
        if (!aligned(dy, in_size(dy_dtype)) || !aligned(h, s) || !aligned(dh, s) || !aligned(dres, s) || !aligned(rstd, 4) ||
            (weight && !aligned(weight, in_size(w_dtype))) || !aligned(ws, 256))
            return MXFP4_ERR_ALIGN;
        if (dres && dh == dres && lddh != lddr) return MXFP4_ERR_ARG;
        if (dweight && ws_bytes < norm_backward_workspace_bytes(rows, cols)) return MXFP4_ERR_WORKSPACE;
    }
    const mxfp4_status_t dev = check_device();
    if (dev != MXFP4_OK) return dev;
    const NormBackward p{{dy, lddy}, {dres, lddr}, {h, ldh}, weight, dy_dtype == MXFP4_IN_F32, stream_dtype == MXFP4_IN_F32,
                         w_dtype == MXFP4_IN_F32, dw_dtype == MXFP4_OUT_F32, rstd, rows, cols, {dh, lddh}, dweight};
    return from_hip(launch_norm_backward(p, ws, static_cast<hipStream_t>(stream)));
}

mxfp4_status_t mxfp4_swiglu_forward(const void *gate, int64_t ldg, const void *up, int64_t ldu, mxfp4_dtype_t dtype,
                                    int64_t rows, int64_t cols, void *a, mxfp4_out_dtype_t a_dtype, int64_t lda, uint8_t *q1,
                                    int64_t ldq1, uint8_t *s1, int64_t lds1, uint8_t *q0, int64_t ldq0, uint8_t *s0,
                                    int64_t lds0, void *stream)
{
    if (!valid_in(dtype) || (a && !valid_out(a_dtype))) return MXFP4_ERR_ARG;
    if (!in_range(rows, 0, kMaxDim) || !in_range(cols, 0, kMaxDim) || tiles(rows, cols) > kLayerTiles) return MXFP4_ERR_SHAPE;
    if (!stride_ok(ldg, rows, cols) || !stride_ok(ldu, rows, cols) || (a && !stride_ok(lda, rows, cols))) return MXFP4_ERR_ARG;
    if (rows == 0 || cols == 0) return MXFP4_OK;
    if (!gate || !up) return MXFP4_ERR_NULL;
    const Fp8Out out1{q1, ldq1, s1, lds1}, out0{q0, ldq0, s0, lds0};
    if (mxfp4_status_t e = check_both(out1, out0, rows, cols)) return e;
    if (!aligned(gate, in_size(dtype)) || !aligned(up, in_size(dtype)) || (a && !aligned(a, out_size(a_dtype)))) return MXFP4_ERR_ALIGN;
    // in place the rows have to be the same ones
    if (a && ((a == gate && lda != ldg) || (a == up && lda != ldu) || ((a == gate || a == up) && out_size(a_dtype) != in_size(dtype))))
        return MXFP4_ERR_ARG;
    if (!a && !q1 && !q0) return MXFP4_OK;
    const mxfp4_status_t dev = check_device();
    if (dev != MXFP4_OK) return dev;
    Gate p{};
    p.g = {gate, ldg};
    p.u = {up, ldu};
    p.f32 = dtype == MXFP4_IN_F32;
    p.out_f32 = a_dtype == MXFP4_OUT_F32;
    p.rows = rows;
    p.cols = cols;
    p.out[0] = {a, lda};
    p.q1[0] = out1;
    p.q0[0] = out0;
    return from_hip(launch_gate(p, static_cast<hipStream_t>(stream)));
}

mxfp4_status_t mxfp4_swiglu_backward(const void *da, mxfp4_dtype_t da_dtype, int64_t ldda, const void *gate, int64_t ldg,
                                     const void *up, int64_t ldu, mxfp4_dtype_t dtype, int64_t rows, int64_t cols, void *dgate,
                                     int64_t lddg, void *dup, int64_t lddu, mxfp4_out_dtype_t out_dtype, uint8_t *q1_gate,
                                     uint8_t *q1_up, int64_t ldq1, uint8_t *s1_gate, uint8_t *s1_up, int64_t lds1,
                                     uint8_t *q0_gate, uint8_t *q0_up, int64_t ldq0, uint8_t *s0_gate, uint8_t *s0_up,
                                     int64_t lds0, void *stream)
{
    if (!valid_in(dtype) || !valid_in(da_dtype) || ((dgate || dup) && !valid_out(out_dtype))) return MXFP4_ERR_ARG;
    if (!in_range(rows, 0, kMaxDim) || !in_range(cols, 0, kMaxDim) || tiles(rows, cols) > kLayerTiles) return MXFP4_ERR_SHAPE;
    if (!stride_ok(ldda, rows, cols) || !stride_ok(ldg, rows, cols) || !stride_ok(ldu, rows, cols) || (dgate && !stride_ok(lddg, rows, cols)) ||
        (dup && !stride_ok(lddu, rows, cols)))
        return MXFP4_ERR_ARG;
    if (rows == 0 || cols == 0) return MXFP4_OK;
    if (!da || !gate || !up) return MXFP4_ERR_NULL;
    const Fp8Out g1{q1_gate, ldq1, s1_gate, lds1}, u1{q1_up, ldq1, s1_up, lds1}, g0{q0_gate, ldq0, s0_gate, lds0},
        u0{q0_up, ldq0, s0_up, lds0};
    if (mxfp4_status_t e = check_both(g1, g0, rows, cols)) return e;
    if (mxfp4_status_t e = check_both(u1, u0, rows, cols)) return e;
    if (!aligned(da, in_size(da_dtype)) || !aligned(gate, in_size(dtype)) || !aligned(up, in_size(dtype)) ||
        (dgate && !aligned(dgate, out_size(out_dtype))) || (dup && !aligned(dup, out_size(out_dtype))))
        return MXFP4_ERR_ALIGN;
    // in place the rows have to be the same ones
    const auto clash = [&](const void *out, int64_t ld) {
        return out && ((out == da && (ld != ldda || out_size(out_dtype) != in_size(da_dtype))) ||
                       (out == gate && (ld != ldg || out_size(out_dtype) != in_size(dtype))) ||
                       (out == up && (ld != ldu || out_size(out_dtype) != in_size(dtype))));
    };
    if (clash(dgate, lddg) || clash(dup, lddu) || (dgate && dgate == dup)) return MXFP4_ERR_ARG;
    if (!dgate && !dup && !q1_gate && !q1_up && !q0_gate && !q0_up) return MXFP4_OK;
    const mxfp4_status_t dev = check_device();
    if (dev != MXFP4_OK) return dev;
    const Gate p{{da, ldda}, {gate, ldg}, {up, ldu}, da_dtype == MXFP4_IN_F32, dtype == MXFP4_IN_F32, out_dtype == MXFP4_OUT_F32,
                 rows, cols, {{dgate, lddg}, {dup, lddu}}, {g1, u1}, {g0, u0}};
    return from_hip(launch_gate(p, static_cast<hipStream_t>(stream)));
}

size_t mxfp4_grad_norm_workspace_bytes(const mxfp4_grad_t *grads, int64_t n)
{
    size_t need = 0;
    guarded([&] {
        std::vector<GradItem> items;
        const mxfp4_status_t e = list_grads(grads, n, false, items);
        if (e == MXFP4_OK) need = grad_norm_workspace_bytes(items.data(), (int64_t)items.size());
        return e;
    });
    return need;
}

mxfp4_status_t mxfp4_grad_norm(const mxfp4_grad_t *grads, int64_t n, void *ws, size_t ws_bytes, double *sum_sq, float *norm,
                               void *stream)
{
    return guarded([&] {
        std::vector<GradItem> items;
        if (mxfp4_status_t e = list_grads(grads, n, false, items)) return e;
        if (!sum_sq && !norm) return MXFP4_OK;
        if (!ws) return MXFP4_ERR_NULL;
        if (!aligned(sum_sq, 8) || !aligned(norm, 4) || !aligned(ws, 256)) return MXFP4_ERR_ALIGN;
        if (ws_bytes < grad_norm_workspace_bytes(items.data(), (int64_t)items.size())) return MXFP4_ERR_WORKSPACE;
        const mxfp4_status_t dev = check_device();
        if (dev != MXFP4_OK) return dev;
        return from_hip(launch_grad_norm(items.data(), (int64_t)items.size(), ws, sum_sq, norm, static_cast<hipStream_t>(stream)));
    });
}

mxfp4_status_t mxfp4_grad_scale(const mxfp4_grad_t *grads, int64_t n, const double *sum_sq, float max_norm, float eps,
                                float *norm, void *stream)
{
    return guarded([&] {
        if (!small_finite(max_norm) || max_norm == 0.0f || !small_finite(eps)) return MXFP4_ERR_ARG;
        std::vector<GradItem> items;
        if (mxfp4_status_t e = list_grads(grads, n, true, items)) return e;
        if (items.empty() && !norm) return MXFP4_OK;
        if (!sum_sq) return MXFP4_ERR_NULL;
        if (!aligned(sum_sq, 8) || !aligned(norm, 4)) return MXFP4_ERR_ALIGN;
        const mxfp4_status_t dev = check_device();
        if (dev != MXFP4_OK) return dev;
        return from_hip(launch_grad_scale(items.data(), (int64_t)items.size(), sum_sq, max_norm, eps, norm, static_cast<hipStream_t>(stream)));
    });
}

mxfp4_status_t mxfp4_grad_clip(const mxfp4_grad_t *grads, int64_t n, float max_norm, float eps, void *ws, size_t ws_bytes,
                               float *norm, void *stream)
{
    return guarded([&] {
        if (!small_finite(max_norm) || max_norm == 0.0f || !small_finite(eps)) return MXFP4_ERR_ARG;
        std::vector<GradItem> items;
        if (mxfp4_status_t e = list_grads(grads, n, true, items)) return e;
        if (items.empty() && !norm) return MXFP4_OK;
        if (!ws) return MXFP4_ERR_NULL;
        if (!aligned(norm, 4) || !aligned(ws, 256)) return MXFP4_ERR_ALIGN;
        if (ws_bytes < grad_norm_workspace_bytes(items.data(), (int64_t)items.size())) return MXFP4_ERR_WORKSPACE;
        const mxfp4_status_t dev = check_device();
        if (dev != MXFP4_OK) return dev;
        return from_hip(launch_grad_clip(items.data(), (int64_t)items.size(), max_norm, eps, ws, norm, static_cast<hipStream_t>(stream)));
    });
}

}  // extern "C"
