// RMS norm of a residual stream: the addition of a branch, the norm, and its result in 8 bits; and its gradient.
//
//   h = x + r (rounded to the stream's type),  rstd = 1 / sqrt(mean_k h_k^2 + eps),  y_k = (h_k rstd) w_k
//   dh = rstd u - h rstd^3 mean_k(u_k h_k) + dres with u_k = dy_k w_k;  dw_k = sum over the rows of dy_k h_k rstd
//
// A row's squares are summed in 64 bits (the square of an FP32 value is exact there and cannot overflow), everything else
// is FP32.
#include <algorithm>

#include "internal.h"
#include "layer_device.h"

namespace mx {
namespace {

// 1 / sqrt(m): the hardware's estimate (2^-23) and one Newton step; 0 and infinity have none
__device__ __forceinline__ float rsqrt64(double m)
{
    const double y = __builtin_amdgcn_rsq(m);
    const double e = fma(-m * y, y, 1.0);
    return m > 0.0 && m < __builtin_inf() ? (float)fma(0.5 * y, e, y) : (float)y;
}

// ------------------------------------------------------------------------------- forward ------
struct ForwardArgs {
    NormForward p;
    double inv_cols;
};

// TPR threads work a row of at most 8 C TPR values, held in registers from the load to the codes.
template <bool XF32, bool SF32, bool RES, bool RAGGED, int TPR, int C>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_forward_kernel(ForwardArgs args)
{
    constexpr int kThreads = TPR < 256 ? 256 : TPR, kRows = kThreads / TPR, kWaves = TPR / 64;
    __shared__ double part[2][kWaves];
    const NormForward &p = args.p;
    const int lane = (int)threadIdx.x % TPR;
    float w[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (p.w) {
            load_any<RAGGED>(p.w_f32, p.w, (c * TPR + lane) * 8, p.cols, w[c]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[c][e] = 1.0f;
        }
    }
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * kRows + (int)threadIdx.x / TPR; row < p.rows;
         row += (int64_t)gridDim.x * kRows) {
        Raw8<XF32> x[C];
        Raw8<SF32> s[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
            x[c] = load_raw<XF32, RAGGED>(at<XF32>(p.x.p, row * p.x.ld), (c * TPR + lane) * 8, p.cols);
        if constexpr (RES) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                s[c] = load_raw<SF32, RAGGED>(at<SF32>(p.r.p, row * p.r.ld), (c * TPR + lane) * 8, p.cols);
        }
        float h[C][8];
        double sum = 0.0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            x[c].get(h[c]);
            if constexpr (RES) {
                float r[8];
                s[c].get(r);
#pragma unroll
                for (int e = 0; e < 8; ++e) r[e] += h[c][e];
                s[c].set(r);
                s[c].get(h[c]);
                if (p.h.p) store_raw<SF32, RAGGED>(s[c], at<SF32>(p.h.p, row * p.h.ld), (c * TPR + lane) * 8, p.cols);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fma((double)h[c][e], (double)h[c][e], sum);
        }
        sum = wave_sum(sum);
        if constexpr (kWaves > 1) {
            // one barrier a row: the next row's sums go to the other half
            if ((lane & 63) == 0) part[turn][lane >> 6] = sum;
            __syncthreads();
            sum = part[turn][0];
#pragma unroll
            for (int i = 1; i < kWaves; ++i) sum += part[turn][i];
            turn ^= 1;
        }
        const float rstd = rsqrt64(fma(sum, args.inv_cols, (double)p.eps));
        if (p.rstd && lane == 0) p.rstd[row] = rstd;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t col = (c * TPR + lane) * 8;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = h[c][e] * rstd * w[c][e];
            if (p.y.p)
                store_any<RAGGED>(p.y_f32, y, p.y_f32 ? at<true>(p.y.p, row * p.y.ld) : at<false>(p.y.p, row * p.y.ld), col, p.cols);
            if (p.q1.q) store_row_codes(p.q1, row, col, p.cols, y);
        }
    }
}

// Rows of any length: a workgroup reads each twice, the second time from the caches if they hold it.
template <bool XF32, bool SF32, bool RES>
__global__ __launch_bounds__(1024) void norm_forward_long_kernel(ForwardArgs args)
{
    __shared__ double part[2][16];
    const NormForward &p = args.p;
    const int tid = threadIdx.x;
    // a whole number of blocks of 128, so that no lane of a block leaves the loop before the others
    const int64_t padded = (p.cols + 127) / 128 * 128;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const void *x = at<XF32>(p.x.p, row * p.x.ld), *r = RES ? at<SF32>(p.r.p, row * p.r.ld) : nullptr;
        const auto sums = [&](int64_t col) {
            Raw8<SF32> s;
            if constexpr (RES) {
                float a[8], b[8];
                load_raw<XF32, true>(x, col, p.cols).get(a);
                load_raw<SF32, true>(r, col, p.cols).get(b);
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] += b[e];
                s.set(a);
            } else {
                s = load_raw<SF32, true>(x, col, p.cols);
            }
            return s;
        };
        void *kept = RES && p.h.p ? at<SF32>(p.h.p, row * p.h.ld) : nullptr;
        double sum = 0.0;
        for (int64_t col = 8 * tid; col < padded; col += 8 * 1024) {
            const Raw8<SF32> s = sums(col);
            if (kept) store_raw<SF32, true>(s, kept, col, p.cols);
            float h[8];
            s.get(h);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fma((double)h[e], (double)h[e], sum);
        }
        sum = wave_sum(sum);
        if ((tid & 63) == 0) part[turn][tid >> 6] = sum;
        __syncthreads();
        sum = part[turn][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) sum += part[turn][i];
        turn ^= 1;
        const float rstd = rsqrt64(fma(sum, args.inv_cols, (double)p.eps));
        if (p.rstd && tid == 0) p.rstd[row] = rstd;
        if (!p.y.p && !p.q1.q) continue;
        for (int64_t col = 8 * tid; col < padded; col += 8 * 1024) {
            // where h is kept, x or r may have been it: what this thread has written is read back
            float h[8], w[8];
            if (kept)
                load_raw<SF32, true>(kept, col, p.cols).get(h);
            else
                sums(col).get(h);
            if (p.w) {
                load_any<true>(p.w_f32, p.w, col, p.cols, w);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = 1.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = h[e] * rstd * w[e];
            if (p.y.p)
                store_any<true>(p.y_f32, h, p.y_f32 ? at<true>(p.y.p, row * p.y.ld) : at<false>(p.y.p, row * p.y.ld), col, p.cols);
            if (p.q1.q) store_row_codes(p.q1, row, col, p.cols, h);
        }
    }
}

// The codes along the columns, in tiles: a block's 128 rows need their rstd first.
template <bool SF32, bool RAGGED>
__global__ __launch_bounds__(512) void norm_columns_kernel(NormForward p, Rows h, int tiles_n)
{
    __shared__ TileShared sh;
    const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
    const int64_t tm = blockIdx.x / (unsigned)tiles_n, tn = blockIdx.x % (unsigned)tiles_n;
    const int64_t row0 = tm * 128 + 4 * rg, col0 = tn * 128 + 8 * cg;
    Raw8<SF32> raw[4];
    float rstd[4], w[8], v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool in = row0 + i < p.rows;
        raw[i].zero();
        if (in) raw[i] = load_raw<SF32, RAGGED>(at<SF32>(h.p, (row0 + i) * h.ld), col0, p.cols);
        rstd[i] = in ? p.rstd[row0 + i] : 0.0f;
    }
    if (p.w) {
        load_any<RAGGED>(p.w_f32, p.w, col0, p.cols, w);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        raw[i].get(v[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = row0 + i < p.rows ? v[i][e] * rstd[i] * w[e] : 0.0f;
    }
    store_tile_columns(p.q0, tm, tn, p.cols, v, sh);
}

template <bool XF32, bool SF32, bool RES, bool RAGGED, int TPR, int C>
hipError_t run_forward(const ForwardArgs &args, hipStream_t stream)
{
    constexpr int kThreads = TPR < 256 ? 256 : TPR, kRows = kThreads / TPR;
    const int64_t blocks = std::min<int64_t>((args.p.rows + kRows - 1) / kRows, (int64_t)1 << 20);
    return launch(norm_forward_kernel<XF32, SF32, RES, RAGGED, TPR, C>, dim3((unsigned)blocks), dim3(kThreads), 0, stream, args);
}
template <bool XF32, bool SF32, bool RES, bool RAGGED>
hipError_t pick_forward(const ForwardArgs &args, hipStream_t stream)
{
    const int64_t cols = args.p.cols;
    if (cols <= 512) return run_forward<XF32, SF32, RES, RAGGED, 64, 1>(args, stream);
    if (cols <= 1024) return run_forward<XF32, SF32, RES, RAGGED, 64, 2>(args, stream);
    if (cols <= 2048) return run_forward<XF32, SF32, RES, RAGGED, 256, 1>(args, stream);
    if (cols <= 4096) return run_forward<XF32, SF32, RES, RAGGED, 256, 2>(args, stream);
    if (cols <= 8192) return run_forward<XF32, SF32, RES, RAGGED, 512, 2>(args, stream);
    if (cols <= 16384) return run_forward<XF32, SF32, RES, RAGGED, 1024, 2>(args, stream);
    const int64_t blocks = std::min<int64_t>(args.p.rows, (int64_t)1 << 20);
    return launch(norm_forward_long_kernel<XF32, SF32, RES>, dim3((unsigned)blocks), dim3(1024), 0, stream, args);
}
template <bool XF32, bool SF32, bool RES>
hipError_t forward(const ForwardArgs &args, hipStream_t stream)
{
    return args.p.cols % 8 ? pick_forward<XF32, SF32, RES, true>(args, stream) : pick_forward<XF32, SF32, RES, false>(args, stream);
}

// ------------------------------------------------------------------------------- backward -----
constexpr int kGradBlocks = 512;   // most workgroups, and so partial sums of dw

struct BackwardArgs {
    NormBackward p;
    float *part;            // [gridDim.x][cols]
    float inv_cols;
    int64_t rows_per_block;
};

template <bool BF32, bool SF32, int C>
struct GradRow {
    Raw8<BF32> dy[C];
    Raw8<SF32> h[C], dres[C];
    float rstd;

    template <bool RAGGED, int TPR>
    __device__ __forceinline__ void load(const NormBackward &p, int64_t row, int64_t end, int lane)
    {
        const bool in = row < end;
        rstd = in ? p.rstd[row] : 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t col = in ? (c * TPR + lane) * 8 : p.cols;      // behind the row: zeros
            dy[c] = load_raw<BF32, RAGGED>(at<BF32>(p.dy.p, row * p.dy.ld), col, p.cols);
            h[c] = load_raw<SF32, RAGGED>(at<SF32>(p.h.p, row * p.h.ld), col, p.cols);
            dres[c] = load_raw<SF32, RAGGED>(at<SF32>(p.dres.p, row * p.dres.ld), p.dres.p ? col : p.cols, p.cols);
        }
    }
};

// A workgroup works rows_per_block rows, ROWS of them at a time in TPR threads each, and keeps its sum of dw in registers until
// the end. With eight values a thread (C = 1) the next rows' loads are under way meanwhile: at 8192 x 4096 the kernel and the
// joining of dw take 56 us with them, 75 with 16 values a thread in 256 and no such loads (58 with them, in 162 registers).
template <bool BF32, bool SF32, bool RAGGED, int TPR, int C, int ROWS>
__global__ __launch_bounds__(TPR *ROWS) void norm_backward_kernel(BackwardArgs args)
{
    constexpr int kWaves = TPR / 64;
    __shared__ float part[2][ROWS][kWaves];
    __shared__ float sums[ROWS > 1 ? TPR * 8 : 1];
    const NormBackward &p = args.p;
    const int lane = (int)threadIdx.x % TPR, slot = (int)threadIdx.x / TPR;
    float w[C][8], dw[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (p.w) {
            load_any<RAGGED>(p.w_f32, p.w, (c * TPR + lane) * 8, p.cols, w[c]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[c][e] = 1.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[c][e] = 0.0f;
    }
    const int64_t first = (int64_t)blockIdx.x * args.rows_per_block, end = min(first + args.rows_per_block, p.rows);
    GradRow<BF32, SF32, C> next;
    if constexpr (C == 1) next.template load<RAGGED, TPR>(p, first + slot, end, lane);
    int turn = 0;
    for (int64_t base = first; base < end; base += ROWS) {
        const int64_t row = base + slot;
        if constexpr (C > 1) next.template load<RAGGED, TPR>(p, row, end, lane);
        GradRow<BF32, SF32, C> r = next;
        if constexpr (C == 1) next.template load<RAGGED, TPR>(p, row + ROWS, end, lane);
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float a[8], b[8];
            r.dy[c].get(a);
            r.h[c].get(b);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = b[e] * r.rstd;
                dw[c][e] = fmaf(a[e], n, dw[c][e]);
                sum = fmaf(a[e] * w[c][e], n, sum);
            }
        }
        sum = wave_sum(sum);
        if constexpr (kWaves > 1) {
            if ((lane & 63) == 0) part[turn][slot][lane >> 6] = sum;
            __syncthreads();
            sum = part[turn][slot][0];
#pragma unroll
            for (int i = 1; i < kWaves; ++i) sum += part[turn][slot][i];
            turn ^= 1;
        }
        if (row >= end) continue;
        const float mean = sum * args.inv_cols;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float a[8], b[8], d[8];
            r.dy[c].renew();
            r.h[c].renew();
            r.dy[c].get(a);
            r.h[c].get(b);
            r.dres[c].get(d);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = fmaf(fmaf(-(b[e] * r.rstd), mean, a[e] * w[c][e]), r.rstd, d[e]);
            Raw8<SF32> out;
            out.set(d);
            store_raw<SF32, RAGGED>(out, at<SF32>(p.dh.p, row * p.dh.ld), (c * TPR + lane) * 8, p.cols);
        }
    }
    if (!p.dw) return;
    // the row groups' sums, added in their order through the LDS, chunk by chunk
    float *to = args.part + (int64_t)blockIdx.x * p.cols;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if constexpr (ROWS > 1) {
            for (int k = 0; k < ROWS; ++k) {
                if (slot == k) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float *at = &sums[e * TPR + lane];
                        *at = k ? *at + dw[c][e] : dw[c][e];
                    }
                }
                __syncthreads();
            }
            if (slot == 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) dw[c][e] = sums[e * TPR + lane];
            }
            __syncthreads();
        }
        if (slot == 0) store_any<RAGGED>(true, dw[c], to, (c * TPR + lane) * 8, p.cols);
    }
}

// Rows of any length: read twice, the sums of dw kept in the workspace.
template <bool BF32, bool SF32>
__global__ __launch_bounds__(1024) void norm_backward_long_kernel(BackwardArgs args)
{
    __shared__ float part[2][16];
    const NormBackward &p = args.p;
    const int tid = threadIdx.x;
    float *dw = args.part + (int64_t)blockIdx.x * p.cols;
    const int64_t first = (int64_t)blockIdx.x * args.rows_per_block, end = min(first + args.rows_per_block, p.rows);
    int turn = 0;
    for (int64_t row = first; row < end; ++row) {
        const void *dy = at<BF32>(p.dy.p, row * p.dy.ld), *h = at<SF32>(p.h.p, row * p.h.ld);
        const float rstd = p.rstd[row];
        float sum = 0.0f;
        for (int64_t col = 8 * tid; col < p.cols; col += 8 * 1024) {
            float a[8], b[8], w[8], d[8];
            load_raw<BF32, true>(dy, col, p.cols).get(a);
            load_raw<SF32, true>(h, col, p.cols).get(b);
            if (p.w) load_any<true>(p.w_f32, p.w, col, p.cols, w);
            if (p.dw && row != first) load_any<true>(true, dw, col, p.cols, d);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = b[e] * rstd;
                sum = fmaf(p.w ? a[e] * w[e] : a[e], n, sum);
                d[e] = row != first ? fmaf(a[e], n, d[e]) : a[e] * n;
            }
            if (p.dw) store_any<true>(true, d, dw, col, p.cols);
        }
        sum = wave_sum(sum);
        if ((tid & 63) == 0) part[turn][tid >> 6] = sum;
        __syncthreads();
        sum = part[turn][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) sum += part[turn][i];
        turn ^= 1;
        const float mean = sum * args.inv_cols;
        for (int64_t col = 8 * tid; col < p.cols; col += 8 * 1024) {
            float a[8], b[8], w[8], d[8] = {};
            load_raw<BF32, true>(dy, col, p.cols).get(a);
            load_raw<SF32, true>(h, col, p.cols).get(b);
            if (p.w) load_any<true>(p.w_f32, p.w, col, p.cols, w);
            if (p.dres.p) load_raw<SF32, true>(at<SF32>(p.dres.p, row * p.dres.ld), col, p.cols).get(d);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                d[e] = fmaf(fmaf(-(b[e] * rstd), mean, p.w ? a[e] * w[e] : a[e]), rstd, d[e]);
            Raw8<SF32> out;
            out.set(d);
            store_raw<SF32, true>(out, at<SF32>(p.dh.p, row * p.dh.ld), col, p.cols);
        }
    }
}

// dw: the workgroups' sums, in a fixed order: 32 columns a workgroup, 32 shares of the sums
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float *part, int count, int64_t cols, void *dw, int f32)
{
    __shared__ float sums[32][32 + 1];
    const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (col < cols) {
#pragma unroll 8
        for (int i = share; i < count; i += 32) sum += part[(int64_t)i * cols + col];
    }
    sums[share][lane] = sum;
    __syncthreads();
    if (share || col >= cols) return;
    for (int i = 1; i < 32; ++i) sum += sums[i][lane];
    if (f32)
        static_cast<float *>(dw)[col] = sum;
    else
        static_cast<uint16_t *>(dw)[col] = (uint16_t)bf16_pair(sum, 0.0f);
}

int64_t grad_blocks(int64_t rows) { return std::min<int64_t>(rows, kGradBlocks); }

template <bool BF32, bool SF32, bool RAGGED>
hipError_t pick_backward(const BackwardArgs &args, unsigned blocks, hipStream_t stream)
{
    const int64_t cols = args.p.cols;
    const auto run = [&](auto kernel, int threads) { return launch(kernel, dim3(blocks), dim3(threads), 0, stream, args); };
    if (cols <= 512) return run(norm_backward_kernel<BF32, SF32, RAGGED, 64, 1, 8>, 512);
    if (cols <= 1024) return run(norm_backward_kernel<BF32, SF32, RAGGED, 128, 1, 4>, 512);
    if (cols <= 2048) return run(norm_backward_kernel<BF32, SF32, RAGGED, 256, 1, 2>, 512);
    if (cols <= 4096) return run(norm_backward_kernel<BF32, SF32, RAGGED, 512, 1, 1>, 512 * 1);
    if (cols <= 8192) return run(norm_backward_kernel<BF32, SF32, RAGGED, 1024, 1, 1>, 1024);
    if (cols <= 16384) return run(norm_backward_kernel<BF32, SF32, RAGGED, 1024, 2, 1>, 1024);
    return run(norm_backward_long_kernel<BF32, SF32>, 1024);
}
template <bool BF32, bool SF32>
hipError_t backward(const BackwardArgs &args, unsigned blocks, hipStream_t stream)
{
    return args.p.cols % 8 ? pick_backward<BF32, SF32, true>(args, blocks, stream)
                           : pick_backward<BF32, SF32, false>(args, blocks, stream);
}

}  // namespace

hipError_t launch_norm_forward(const NormForward &p, hipStream_t stream)
{
    const ForwardArgs args{p, 1.0 / (double)p.cols};
    const bool res = p.r.p != nullptr;
    hipError_t e;
    if (!res)
        e = p.x_f32 ? forward<true, true, false>(args, stream) : forward<false, false, false>(args, stream);
    else if (p.x_f32)
        e = p.s_f32 ? forward<true, true, true>(args, stream) : forward<true, false, true>(args, stream);
    else
        e = p.s_f32 ? forward<false, true, true>(args, stream) : forward<false, false, true>(args, stream);
    if (e != hipSuccess || !p.q0.q) return e;
    const Rows h = res ? Rows{p.h.p, p.h.ld} : p.x;
    const bool f32 = res ? p.s_f32 : p.x_f32, ragged = p.cols % 8 != 0;
    const int64_t tiles_n = (p.cols + 127) / 128;
    const dim3 grid((unsigned)((p.rows + 127) / 128 * tiles_n)), block(512);
    if (f32)
        return ragged ? launch(norm_columns_kernel<true, true>, grid, block, 0, stream, p, h, (int)tiles_n)
                      : launch(norm_columns_kernel<true, false>, grid, block, 0, stream, p, h, (int)tiles_n);
    return ragged ? launch(norm_columns_kernel<false, true>, grid, block, 0, stream, p, h, (int)tiles_n)
                  : launch(norm_columns_kernel<false, false>, grid, block, 0, stream, p, h, (int)tiles_n);
}

size_t norm_backward_workspace_bytes(int64_t rows, int64_t cols)
{
    return (size_t)(grad_blocks(rows) * cols) * sizeof(float);
}

hipError_t launch_norm_backward(const NormBackward &p, void *ws, hipStream_t stream)
{
    // every workgroup has a row, and so every partial sum is written
    const int64_t per = p.rows ? (p.rows + grad_blocks(p.rows) - 1) / grad_blocks(p.rows) : 1, blocks = (p.rows + per - 1) / per;
    if (blocks > 0) {
        const BackwardArgs args{p, static_cast<float *>(ws), (float)(1.0 / (double)p.cols), per};
        hipError_t e;
        if (p.b_f32)
            e = p.s_f32 ? backward<true, true>(args, (unsigned)blocks, stream) : backward<true, false>(args, (unsigned)blocks, stream);
        else
            e = p.s_f32 ? backward<false, true>(args, (unsigned)blocks, stream) : backward<false, false>(args, (unsigned)blocks, stream);
        if (e != hipSuccess) return e;
    }
    if (!p.dw) return hipSuccess;
    return launch(norm_dw_kernel, dim3((unsigned)((p.cols + 31) / 32)), dim3(1024), 0, stream, static_cast<const float *>(ws),
                  (int)blocks, p.cols, p.dw, p.dw_f32 ? 1 : 0);
}

}  // namespace mx
