// The gradients of the RMS norm:
//
//   dh = rstd u - h rstd^3 mean_k(u_k h_k) + dres with u_k = dy_k w_k;  dw_k = sum over the rows of dy_k h_k rstd
//
// in FP32, dh as rstd (u - n mean_k(u_k n_k)) + dres with n = h rstd.
//
// Bound by memory: 8192 x 4096 in bf16 with dres 52 to 54 us for 268 MB (a copy of as much 53), 50 in the rows' kernel and 5 to join dw.
// Small calls are two launches: 16 x 8192 6.6 us, 1024 x 1024 6.9.
#include <algorithm>

#include "internal.h"
#include "layer_device.h"

namespace mx {
namespace {

constexpr int kGradBlocks = 512;   // most workgroups, and so partial sums of dw

struct BackwardArgs {
    NormBackward p;
    float *part;            // [gridDim.x][cols]
    float inv_cols;
    int64_t rows_per_block;
};

template <bool BF32, bool SF32, Ends E, int TPR, int C>
struct GradRow {
    Raw8<BF32> dy[C];
    Raw8<SF32> h[C], dres[C];
    float rstd;

    static __device__ __forceinline__ Eight<E> eight(const NormBackward &p, int c, int lane) { return {(c * TPR + lane) * 8, p.cols}; }

    // A row behind the end is read as the last one, or not at all; settle() makes zeros of it (dh may be dres, and the last row be
    // written meanwhile: nothing of what is read here is used then).
    template <bool NT>
    __device__ __forceinline__ void load(const NormBackward &p, int64_t row, int64_t end, int lane)
    {
        row = min(row, end - 1);
        rstd = p.rstd[row];
        const void *at_dy = at<BF32>(p.dy.p, row * p.dy.ld), *at_h = at<SF32>(p.h.p, row * p.h.ld), *at_dres = at<SF32>(p.dres.p, row * p.dres.ld);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            dy[c] = eight(p, c, lane).template load<BF32, NT>(at_dy);
            h[c] = eight(p, c, lane).template load<SF32, NT>(at_h);
            if (p.dres.p)
                dres[c] = eight(p, c, lane).template load<SF32, NT>(at_dres);
            else
                dres[c].zero();
        }
    }
    __device__ __forceinline__ void settle(const NormBackward &p, bool in, int lane)
    {
        if (!in) rstd = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (const int gone = in ? eight(p, c, lane).gone() : 8) {
                dy[c].drop(gone);
                h[c].drop(gone);
                dres[c].drop(gone);
            }
        }
    }
};

// A workgroup works rows_per_block rows, ROWS of them at a time in TPR threads each, and keeps its sum of dw in registers until
// the end. With eight values a thread (C = 1) the next rows' loads are under way meanwhile: at 8192 x 4096 the kernel and the
// joining of dw take 56 us with them, 75 with 16 values a thread in 256 and no such loads (58 with them, in 162 registers).
template <bool BF32, bool SF32, Ends E, bool NT, int TPR, int C, int ROWS>
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
            load_any<E != kWhole>(p.w_f32, p.w, (c * TPR + lane) * 8, p.cols, w[c]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[c][e] = 1.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[c][e] = 0.0f;
    }
    const int64_t first = (int64_t)blockIdx.x * args.rows_per_block, end = min(first + args.rows_per_block, p.rows);
    GradRow<BF32, SF32, E, TPR, C> next;
    if constexpr (C == 1) next.template load<NT>(p, first + slot, end, lane);
    int turn = 0;
    for (int64_t base = first; base < end; base += ROWS) {
        const int64_t row = base + slot;
        if constexpr (C > 1) next.template load<NT>(p, row, end, lane);
        GradRow<BF32, SF32, E, TPR, C> r = next;
        if constexpr (C == 1)
            if (__builtin_amdgcn_readfirstlane((int)(row + ROWS < end))) next.template load<NT>(p, row + ROWS, end, lane);
        r.settle(p, row < end, lane);
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
            store_raw<SF32, E != kWhole>(out, at<SF32>(p.dh.p, row * p.dh.ld), (c * TPR + lane) * 8, p.cols);
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
        if (slot == 0) store_any<E != kWhole>(true, dw[c], to, (c * TPR + lane) * 8, p.cols);
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

// How the rows are shared out: as many at a time as pick_backward's kernels take, every workgroup having some, so that every
// partial sum is written.
struct Shares {
    int64_t blocks, rows;   // rows of a workgroup, the last one's fewer
};
Shares shares(int64_t rows, int64_t cols)
{
    const int64_t at_once = cols <= 512 ? 8 : cols <= 1024 ? 4 : cols <= 2048 ? 2 : 1;
    const int64_t groups = (rows + at_once - 1) / at_once, each = std::max<int64_t>((groups + kGradBlocks - 1) / kGradBlocks, 1);
    return {(groups + each - 1) / each, each * at_once};
}

template <bool BF32, bool SF32, Ends E, bool NT>
hipError_t pick_backward(const BackwardArgs &args, unsigned blocks, hipStream_t stream)
{
    const int64_t cols = args.p.cols;
    const auto run = [&](auto kernel, int threads) { return launch(kernel, dim3(blocks), dim3(threads), 0, stream, args); };
    if (E == kFew || cols <= 512) return run(norm_backward_kernel<BF32, SF32, E, NT, 64, 1, 8>, 512);
    if constexpr (E != kFew) {
        if (cols <= 1024) return run(norm_backward_kernel<BF32, SF32, E, NT, 128, 1, 4>, 512);
        if (cols <= 2048) return run(norm_backward_kernel<BF32, SF32, E, NT, 256, 1, 2>, 512);
        if (cols <= 4096) return run(norm_backward_kernel<BF32, SF32, E, NT, 512, 1, 1>, 512);
        if (cols <= 8192) return run(norm_backward_kernel<BF32, SF32, E, NT, 1024, 1, 1>, 1024);
        if (cols <= 16384) return run(norm_backward_kernel<BF32, SF32, E, NT, 1024, 2, 1>, 1024);
    }
    return run(norm_backward_long_kernel<BF32, SF32>, 1024);
}
// Streaming loads where the call is more than the last cache takes and the stream is bf16 (outputs in new memory; where rows start at
// multiples of 16 bytes, and where not): 8192 x 4096 (268 MB) 61 -> 58 us and 60 -> 59, with dy in FP32 74 -> 69 and 74 -> 73, 5000 x 8192
// 72 -> 71 and 83 -> 82, 32768 x 1024 58 -> 56 and 58 -> 58; 4096 x 4096 (134 MB) 30 both ways, 2048 x 4096 18 and 23. With an FP32 stream
// 8192 x 8192 takes 189 and 187, and 189 and 192; dy in FP32 as well 8192 x 4096 110 and 112, and 111 and 115. Not for rows that end within
// eight values: a line that two loads share is read twice.
template <bool BF32, bool SF32>
hipError_t backward(const BackwardArgs &args, unsigned blocks, hipStream_t stream)
{
    const NormBackward &p = args.p;
    if (p.cols % 8)
        return p.cols < 8 ? pick_backward<BF32, SF32, kFew, false>(args, blocks, stream) : pick_backward<BF32, SF32, kWithin, false>(args, blocks, stream);
    if constexpr (!SF32) {
        const int64_t bytes = p.rows * p.cols * ((BF32 ? 4 : 2) + (p.dres.p ? 6 : 4));
        if (bytes > kStreamBytes) return pick_backward<BF32, SF32, kWhole, true>(args, blocks, stream);
    }
    return pick_backward<BF32, SF32, kWhole, false>(args, blocks, stream);
}

}  // namespace

size_t norm_backward_workspace_bytes(int64_t rows, int64_t cols)
{
    return (size_t)(shares(rows, cols).blocks * cols) * sizeof(float);
}

hipError_t launch_norm_backward(const NormBackward &p, void *ws, hipStream_t stream)
{
    const auto [blocks, per] = shares(p.rows, p.cols);
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
