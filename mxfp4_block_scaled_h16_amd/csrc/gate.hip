// The gated activation a = silu(g) u and its gradients, in 16 / 32 bits and as 8-bit codes along both axes.
//
//   s = 1 / (1 + exp(-g));  a = g s u
//   du = da g s,  dg = da u s (1 + g (1 - s))
//
// One pass: a workgroup works a tile of 128 x 128 values, which holds whole blocks along both axes.
#include <cfloat>

#include "internal.h"
#include "layer_device.h"

namespace mx {
namespace {

// s = 1 / (1 + e) and 1 - s = e s, e = exp(-g). The hardware's exponential and reciprocal are off by 2^-23 each, and the
// exponent's rounding, |g| 2^-24, is one of e: s and 1 - s are off by at most (8 + 1.3 |g|) 2^-24 of themselves, the larger of the
// two by far less. Below g = -88 e is infinite and s zero, where it is below 2^-126 (1 - s is multiplied with it).
__device__ __forceinline__ float sigmoid(float g, float &e)
{
    e = __builtin_amdgcn_exp2f(g * -1.44269504088896340736f);
    return __builtin_amdgcn_rcpf(1.0f + e);
}

// GRAD: the gradients, from da; DF32: da's type. F32: that of g and u.
template <bool GRAD, bool DF32, bool F32, bool RAGGED, bool NT>
__global__ __launch_bounds__(512, 4) void gate_kernel(Gate p, int tiles_n)
{
    __shared__ TileShared sh;
    const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
    const auto [tm, tn] = tile_of(tiles_n);
    const int64_t row0 = tm * 128 + 4 * rg, col0 = tn * 128 + 8 * cg;
    Raw8<F32> g[4], u[4];
    Raw8<DF32> d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = row0 + i;
        g[i].zero();
        u[i].zero();
        d[i].zero();
        if (row >= p.rows) continue;
        g[i] = load_raw<F32, RAGGED, NT>(at<F32>(p.g.p, row * p.g.ld), col0, p.cols);
        u[i] = load_raw<F32, RAGGED, NT>(at<F32>(p.u.p, row * p.u.ld), col0, p.cols);
        if constexpr (GRAD) d[i] = load_raw<DF32, RAGGED, NT>(at<DF32>(p.da.p, row * p.da.ld), col0, p.cols);
    }
    float v[GRAD ? 2 : 1][4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a[8], b[8], c[8];
        g[i].get(a);
        u[i].get(b);
        if constexpr (GRAD) d[i].get(c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float x;
            const float s = sigmoid(a[e], x);
            if constexpr (GRAD) {
                const float t = fminf(x, FLT_MAX) * s;
                v[0][i][e] = c[e] * b[e] * (s * fmaf(a[e], t, 1.0f));
                v[1][i][e] = c[e] * (a[e] * s);
                // both now, while the inputs leave their registers: formed where they are used, they hold 186 instead
                asm volatile("" : "+v"(v[1][i][e]));
            } else {
                v[0][i][e] = a[e] * s * b[e];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < (GRAD ? 2 : 1); ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = row0 + i;
            if (row >= p.rows) break;
            if (p.out[k].p)
                store_any<RAGGED>(p.out_f32, v[k][i],
                                  p.out_f32 ? at<true>(p.out[k].p, row * p.out[k].ld) : at<false>(p.out[k].p, row * p.out[k].ld),
                                  col0, p.cols);
            if (p.q1[k].q) store_row_codes(p.q1[k], row, col0, p.cols, v[k][i]);
        }
        if (p.q0[k].q) store_tile_columns(p.q0[k], tm, tn, p.cols, v[k], sh);
    }
}

// Where inputs and outputs are more than the last cache holds, the inputs' loads do not stay in it: 8192 x 14336 (704 MB) 142 ->
// 121 us, 4096 x 14336 71 -> 63; where they fit, the input is mostly still there from the product that wrote it:
// 2048 x 14336 (176 MB) 30 us, and 34 with such loads.
constexpr int64_t kLastCache = (int64_t)256 << 20;

template <bool GRAD, bool DF32, bool F32>
hipError_t run(const Gate &p, hipStream_t stream)
{
    const int64_t tiles_n = (p.cols + 127) / 128;
    const dim3 grid((unsigned)((p.rows + 127) / 128 * tiles_n)), block(512);
    int64_t bytes = (F32 ? 8 : 4) + (GRAD ? DF32 ? 4 : 2 : 0);
    for (int k = 0; k < 2; ++k) bytes += (p.out[k].p ? p.out_f32 ? 4 : 2 : 0) + (p.q1[k].q ? 1 : 0) + (p.q0[k].q ? 1 : 0);
    if (p.cols % 8) return launch(gate_kernel<GRAD, DF32, F32, true, false>, grid, block, 0, stream, p, (int)tiles_n);
    return p.rows * p.cols > kLastCache / bytes ? launch(gate_kernel<GRAD, DF32, F32, false, true>, grid, block, 0, stream, p, (int)tiles_n)
                                                : launch(gate_kernel<GRAD, DF32, F32, false, false>, grid, block, 0, stream, p, (int)tiles_n);
}

}  // namespace

hipError_t launch_gate(const Gate &p, hipStream_t stream)
{
    if (!p.da.p) return p.f32 ? run<false, true, true>(p, stream) : run<false, false, false>(p, stream);
    if (p.da_f32) return p.f32 ? run<true, true, true>(p, stream) : run<true, true, false>(p, stream);
    return p.f32 ? run<true, false, true>(p, stream) : run<true, false, false>(p, stream);
}

}  // namespace mx
