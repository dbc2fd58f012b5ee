// The gated activation a = silu(g) u and its gradients, in 16 / 32 bits and as 8-bit codes along both axes.
//
//   s = 1 / (1 + exp(-g));  a = g s u
//   du = da g s,  dg = da u s (1 + g (1 - s))
//
// One pass: a workgroup works a tile of 128 x 128 values, which holds whole blocks along both axes, in registers.
//
// Bound by memory. 8192 x 14336 in bf16 with codes along both axes: forward 121 to 125 us (704 MB, 5.7 TB/s; a kernel that only
// reads and writes as many streams 117 to 134), the gradient 236 (1174 MB, 5.0 TB/s; such a kernel 206 to 222). The scale bytes, one
// to a line, are 11 us of the gradient's, the turning of the codes 2; more wavefronts (1024 threads of half the values, up
// to eight a SIMD) made it 266, one pass through the LDS for both gradients no difference.
#include "internal.h"
#include "layer_device.h"

namespace mx {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;                                   // ln 2, rounded
constexpr float kLn2Low = (float)(0.69314718055994530942 - (double)kLn2);        // and what the rounding left

// s = 1 / (1 + e) and 1 - s = e s, e = exp(-g). exp2's argument k = -g log2(e) is rounded by up to |k| 2^-24, which the exponential would
// multiply by: -g = k ln 2 + r gives r, and e = 2^k (1 + r). The reciprocal is the hardware's with a Newton step, whose remainder 1 - s -
// e s knows e as it was before 1 + e rounded it. In units of 2^-24 of the value at most: e 3.1 (the hardware's 2, the last sum's 1), s
// 4.6 (e's, half for 1 - s, the last sum's 1), 1 - s 5.6; measured 3.5 for g s. 11 operations where the hardware's functions alone are 4, which
// are off by up to 16 at g = -16 and 65 at -80; 8192 x 14336 takes 121 us with either, the gradient 235 and 236, 256 x 512 4.9 instead of 4.2.
// e stays finite, and s is zero from 1 + e = 2^126 on, as the reciprocal has no subnormal results: so an infinite g gives what the
// formulas do, and a NaN, for which e is some number, comes back in the products with g.
__device__ __forceinline__ float sigmoid(float g, float &e)
{
    const float x = __builtin_amdgcn_fmed3f(g, -88.5f, 128.0f);
    const float k = x * -1.44269504088896340736f;
    const float r = fmaf(k, -kLn2Low, fmaf(k, -kLn2, -x));
    e = __builtin_amdgcn_exp2f(k);
    e = fmaf(e, r, e);
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    return fmaf(fmaf(-e, s, 1.0f - s), s, s);
}

// One tile. GRAD: the gradients, from da; DF32: da's type. F32: that of g and u. kWhole: the tile lies inside the matrix, so that
// nothing is checked and a row's address is the one before and a stride: six VALU operations a value fewer in the gradient,
// which the large sizes do not notice, but the small ones do (256 x 512 forward 5.1 -> 4.9 us, the gradient of 1111 x 2001 in
// FP32 17.3 -> 16.6). kWithin, of the forward pass only: all that a thread has at the matrix' ends is read without branches, the
// last row again behind it (1111 x 2001 9.5 -> 8.1 us, in FP32 10.0 -> 8.5); the gradient would spill (17 -> 27). kFew: value by value.
template <bool GRAD, bool DF32, bool F32, bool NT, Ends E>
__device__ __forceinline__ void gate_tile(const Gate &p, int64_t tm, int64_t tn, TileShared &sh)
{
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int64_t row0 = tm * 128 + 4 * rg, col0 = tn * 128 + 8 * cg;
    constexpr bool FULL = E == kWhole;
    // rows that are loaded and formed together: one in FP32 and two in bf16, as more at once take the registers of the values and
    // come no sooner (8192 x 7168 in FP32 with codes along both axes: gradient 200 us, 204 with two rows and 211 with four, forward 122,
    // 121 and 126; 8192 x 14336 in bf16: 235 and 121, with four 236 and 122, with one 236 and 125). At the ends, where a thread
    // may read value by value, all four (the gradient of 1111 x 2001 in FP32 17 us, with two 29: spilled registers)
    constexpr int BATCH = !FULL ? 4 : F32 || DF32 ? 1 : 2;
    const Eight<E> eight(col0, p.cols);
    const void *gp = at<F32>(p.g.p, row0 * p.g.ld), *up = at<F32>(p.u.p, row0 * p.u.ld), *dp = at<DF32>(p.da.p, row0 * p.da.ld);
    float v[GRAD ? 2 : 1][4][8];
#pragma unroll
    for (int first = 0; first < 4; first += BATCH) {
        Raw8<F32> g[BATCH], u[BATCH];
        Raw8<DF32> d[BATCH];
        if (first) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int i = first + j;
            if constexpr (FULL) {
                g[j].template load<NT>(at<F32>(gp, i * p.g.ld + col0));
                u[j].template load<NT>(at<F32>(up, i * p.u.ld + col0));
                if constexpr (GRAD) d[j].template load<NT>(at<DF32>(dp, i * p.da.ld + col0));
            } else if constexpr (E == kWithin) {
                const int64_t row = min((int64_t)i, p.rows - 1 - row0);
                g[j] = eight.template load<F32, NT>(at<F32>(gp, row * p.g.ld));
                u[j] = eight.template load<F32, NT>(at<F32>(up, row * p.u.ld));
            } else {
                const int64_t cols = row0 + i < p.rows ? p.cols : 0;
                g[j] = load_raw<F32, true, NT>(at<F32>(gp, i * p.g.ld), col0, cols);
                u[j] = load_raw<F32, true, NT>(at<F32>(up, i * p.u.ld), col0, cols);
                if constexpr (GRAD) d[j] = load_raw<DF32, true, NT>(at<DF32>(dp, i * p.da.ld), col0, cols);
            }
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int i = first + j;
            if constexpr (E == kWithin) {
                const int gone = row0 + i < p.rows ? eight.gone() : 8;
                if (gone) {
                    g[j].drop(gone);
                    u[j].drop(gone);
                }
            }
            float a[8], b[8], c[8];
            g[j].get(a);
            u[j].get(b);
            if constexpr (GRAD) d[j].get(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float x;
                const float s = sigmoid(a[e], x);
                if constexpr (GRAD) {
                    // s (1 + g (1 - s)) as s + (g s) (1 - s): one rounding less
                    const float f = a[e] * s;
                    v[0][i][e] = c[e] * (b[e] * fmaf(f, x * s, s));
                    v[1][i][e] = c[e] * f;
                    // now, while the inputs leave their registers: formed where it is used, the kernel holds 186 (345 us instead
                    // of 256 at 8192 x 14336)
                    asm volatile("" : "+v"(v[1][i][e]));
                } else {
                    v[0][i][e] = a[e] * s * b[e];
                    asm volatile("" : "+v"(v[0][i][e]));    // likewise: 76 registers instead of 87
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < (GRAD ? 2 : 1); ++k) {
        if (p.out[k].p) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                store_any<!FULL>(p.out_f32, v[k][i],
                                 p.out_f32 ? at<true>(p.out[k].p, (row0 + i) * p.out[k].ld) : at<false>(p.out[k].p, (row0 + i) * p.out[k].ld),
                                 col0, FULL || row0 + i < p.rows ? p.cols : 0);
        }
        if (p.q1[k].q) {
            uint8_t *q = p.q1[k].q + row0 * p.q1[k].ldq + col0, *to = p.q1[k].s + row0 * p.q1[k].lds + tn;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t s;
                const u32x2 w = row_codes(v[k][i], s);
                if (FULL || row0 + i < p.rows) {
                    store_codes<NT>(w, q + i * p.q1[k].ldq);
                    if (cg == 0) to[i * p.q1[k].lds] = (uint8_t)s;
                }
            }
        }
        if (p.q0[k].q) store_tile_columns<false>(p.q0[k], tm, tn, FULL ? INT64_MAX : p.cols, v[k], sh);
    }
}

template <bool GRAD, bool DF32, bool F32, bool NT>
__global__ __launch_bounds__(512, GRAD || F32 ? 4 : 6) void gate_kernel(Gate p, int tiles_n)
{
    __shared__ TileShared sh;
    const auto [tm, tn] = tile_of(tiles_n);
    if ((tm + 1) * 128 <= p.rows && (tn + 1) * 128 <= p.cols)
        gate_tile<GRAD, DF32, F32, NT, kWhole>(p, tm, tn, sh);
    else if (GRAD || p.cols < 8)
        gate_tile<GRAD, DF32, F32, NT, kFew>(p, tm, tn, sh);
    else if constexpr (!GRAD)
        gate_tile<GRAD, DF32, F32, NT, kWithin>(p, tm, tn, sh);
}

// bf16 rows that all start at multiples of 16 bytes (or none: the forward pass has no da)
bool lines(const Rows &r) { return (uintptr_t)r.p % 16 == 0 && r.ld % 8 == 0; }

// Streaming loads, and stores of the codes along the rows, where the call is more than the last cache takes, all of it is bf16 and rows
// start at multiples of 16 bytes (a line that two loads share is read twice): 4096 x 14336 with codes along both axes (352 MB) 74 -> 67 us,
// 8192 x 14336 143 -> 138, the gradient 126 -> 121 and 244 -> 237 (separate matrices, outputs in new memory); at 1024 x 14336 (88 MB)
// 18.6 and 19.7. Such stores of the codes along the columns as well: 151 and 268. Rows that start elsewhere: 8192 x 14336 148 and 159,
// 255 and 261, bf16 results alone 136 and 157, 230 and 260. FP32: 8192 x 7168 122 and 129, 200 and 217.
template <bool GRAD, bool DF32, bool F32>
hipError_t run(const Gate &p, hipStream_t stream)
{
    const int64_t tiles_n = (p.cols + 127) / 128;
    const dim3 grid((unsigned)((p.rows + 127) / 128 * tiles_n)), block(512);
    if constexpr (!DF32 && !F32) {
        int64_t bytes = GRAD ? 6 : 4;
        for (int k = 0; k < 2; ++k) bytes += (p.out[k].p ? p.out_f32 ? 4 : 2 : 0) + (p.q1[k].q ? 1 : 0) + (p.q0[k].q ? 1 : 0);
        if (p.rows * p.cols > kStreamBytes / bytes && lines(p.g) && lines(p.u) && lines(p.da))
            return launch(gate_kernel<GRAD, DF32, F32, true>, grid, block, 0, stream, p, (int)tiles_n);
    }
    return launch(gate_kernel<GRAD, DF32, F32, false>, grid, block, 0, stream, p, (int)tiles_n);
}

}  // namespace

hipError_t launch_gate(const Gate &p, hipStream_t stream)
{
    if (!p.da.p) return p.f32 ? run<false, true, true>(p, stream) : run<false, false, false>(p, stream);
    if (p.da_f32) return p.f32 ? run<true, true, true>(p, stream) : run<true, true, false>(p, stream);
    return p.f32 ? run<true, false, true>(p, stream) : run<true, false, false>(p, stream);
}

}  // namespace mx
