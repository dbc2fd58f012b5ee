// Launchers behind libmxfp4_layer's C ABI (not part of the public interface). Arguments are
// validated by the caller; these pick a kernel and enqueue it.
#pragma once

#include "train_internal.h"   // Fp8Out, kMaxItems, round_up

namespace mx {

// rows of `ld` elements each; p == nullptr: not there
struct Rows {
    const void *p;
    int64_t ld;
};
struct OutRows {
    void *p;
    int64_t ld;
};

// tiles of 128 x 128 that a grid holds, 512 threads each
constexpr int64_t kLayerTiles = kMaxItems / 512;

// A call that reads and writes more than this goes past the caches where it can: the last one holds 256 MB, and something of the
// call before and behind stays in it.
constexpr int64_t kStreamBytes = (int64_t)192 << 20;

// ------------------------------------------------------------------------------- RMS norm -----
struct NormForward {
    Rows x, r;              // r.p == nullptr: h = x
    const void *w;          // nullptr: ones
    bool x_f32, s_f32, w_f32, y_f32;
    int64_t rows, cols;
    float eps;
    OutRows h, y;
    float *rstd;            // required by q0
    Fp8Out q1, q0;          // q0 reads h (x without r)
};
hipError_t launch_norm_forward(const NormForward &p, hipStream_t stream);

struct NormBackward {
    Rows dy, dres, h;       // dres.p may be nullptr
    const void *w;
    bool b_f32, s_f32, w_f32, dw_f32;   // dy; dres, h, dh; w; dw
    const float *rstd;
    int64_t rows, cols;
    OutRows dh;
    void *dw;               // nullptr: not wanted
};
size_t norm_backward_workspace_bytes(int64_t rows, int64_t cols);
hipError_t launch_norm_backward(const NormBackward &p, void *ws, hipStream_t stream);

// ------------------------------------------------------------------------- gated activation ---
struct Gate {
    Rows da, g, u;          // da.p == nullptr: the forward pass
    bool da_f32, f32, out_f32;
    int64_t rows, cols;
    OutRows out[2];         // a, or dgate and dup
    Fp8Out q1[2], q0[2];
};
hipError_t launch_gate(const Gate &p, hipStream_t stream);

// ------------------------------------------------------------------------- gradients' norm ----
struct GradItem {
    const void *g;
    void *out;
    int64_t count;
    bool f32, out_f32;
};
// items of no values are left out by the caller
size_t grad_norm_workspace_bytes(const GradItem *items, int64_t n);
// sum_sq, norm: either may be nullptr
hipError_t launch_grad_norm(const GradItem *items, int64_t n, void *ws, double *sum_sq, float *norm, hipStream_t stream);
hipError_t launch_grad_scale(const GradItem *items, int64_t n, const double *sum_sq, float max_norm, float eps,
                             float *norm, hipStream_t stream);
hipError_t launch_grad_clip(const GradItem *items, int64_t n, float max_norm, float eps, void *ws, float *norm,
                            hipStream_t stream);

}  // namespace mx
