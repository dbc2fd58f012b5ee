// RMS norm of a residual stream: the addition of a branch, the norm, and its result in 8 bits.
//
//   h = x + r (rounded to the stream's type),  rstd = 1 / sqrt(mean_k h_k^2 + eps),  y_k = (h_k rstd) w_k
//
// A row's squares are summed in 64 bits (the square of an FP32 value is exact there and cannot overflow; no time beside the
// loads), everything else is FP32. A row stays in registers from the load to the codes along it. The codes along the columns need
// the rstd of 128 rows, 1 MB of values at 4096 columns, which no workgroup holds: a second kernel reads h again.
//
// Bound by memory. 8192 x 4096 in bf16 with residual and codes along both axes: 57 to 60 us for 268 MB (and 67 MB of h again), 42 in
// the first kernel (5.6 TB/s) and 17 in the second (5.8); a copy of 268 MB takes 53.
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

// TPR threads work a row of at most 8 C TPR values, held in registers from the load to the codes: a wavefront (WAVE; four of them a
// workgroup), or a workgroup of as many wavefronts as the row needs.
template <bool XF32, bool SF32, bool RES, Ends E, bool NT, bool WAVE, int C>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_forward_kernel(ForwardArgs args)
{
    constexpr int kRows = WAVE ? 4 : 1;
    __shared__ double part[2][16];
    const NormForward &p = args.p;
    const int TPR = WAVE ? 64 : (int)blockDim.x, lane = WAVE ? (int)threadIdx.x % 64 : (int)threadIdx.x;
    float w[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (p.w) {
            load_any<E != kWhole>(p.w_f32, p.w, (c * TPR + lane) * 8, p.cols, w[c]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[c][e] = 1.0f;
        }
    }
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * kRows + (WAVE ? (int)threadIdx.x / 64 : 0); row < p.rows;
         row += (int64_t)gridDim.x * kRows) {
        Raw8<XF32> x[C];
        Raw8<SF32> s[C];
        const auto eight = [&](int c) { return Eight<E>((c * TPR + lane) * 8, p.cols); };
        const void *xr = at<XF32>(p.x.p, row * p.x.ld), *rr = at<SF32>(p.r.p, row * p.r.ld);
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = eight(c).template load<XF32, NT>(xr);
        if constexpr (RES) {
#pragma unroll
            for (int c = 0; c < C; ++c) s[c] = eight(c).template load<SF32, NT>(rr);
        }
        if constexpr (E == kWithin) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (const int gone = eight(c).gone()) {
                    x[c].drop(gone);
                    if constexpr (RES) s[c].drop(gone);
                }
            }
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
                if (p.h.p) store_raw<SF32, E != kWhole>(s[c], at<SF32>(p.h.p, row * p.h.ld), (c * TPR + lane) * 8, p.cols);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fma((double)h[c][e], (double)h[c][e], sum);
        }
        sum = wave_sum(sum);
        if constexpr (!WAVE) {
            // one barrier a row: the next row's sums go to the other half
            if ((lane & 63) == 0) part[turn][lane >> 6] = sum;
            __syncthreads();
            sum = part[turn][0];
            for (int i = 1; i < TPR / 64; ++i) sum += part[turn][i];
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
                store_any<E != kWhole>(p.y_f32, y, p.y_f32 ? at<true>(p.y.p, row * p.y.ld) : at<false>(p.y.p, row * p.y.ld), col, p.cols);
            if (p.q1.q) store_row_codes<NT>(p.q1, row, col, p.cols, y);
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
            if (p.q1.q) store_row_codes<false>(p.q1, row, col, p.cols, h);
        }
    }
}

// The codes along the columns, in tiles: a block's 128 rows need their rstd first. kWhole: the tile lies inside the
// matrix. kWithin: what is read at its ends is read without branches, the last row again behind it (1111 x 2001 in FP32, both
// kernels, 14.9 -> 14.6 us, 128 x 4095 in bf16 12.4 -> 10.7, 100 x 60 9.3 -> 8.1). kFew: value by value.
template <bool SF32, bool NT, Ends E>
__device__ __forceinline__ void norm_tile(const NormForward &p, const Rows &h, int64_t tm, int64_t tn, TileShared &sh)
{
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int64_t row0 = tm * 128 + 4 * rg, col0 = tn * 128 + 8 * cg;
    const void *at0 = at<SF32>(h.p, row0 * h.ld);
    constexpr bool FULL = E == kWhole;
    const Eight<E> eight(col0, p.cols);
    Raw8<SF32> raw[4];
    float rstd[4], w[8], v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool in = FULL || row0 + i < p.rows;
        if constexpr (FULL)
            raw[i].template load<false>(at<SF32>(at0, i * h.ld + col0));
        else if constexpr (E == kWithin)
            raw[i] = eight.template load<SF32, false>(at<SF32>(at0, min((int64_t)i, p.rows - 1 - row0) * h.ld));
        else
            raw[i] = load_raw<SF32, true>(at<SF32>(at0, i * h.ld), col0, in ? p.cols : 0);
        rstd[i] = in ? p.rstd[row0 + i] : 0.0f;
    }
    if (p.w) {
        load_any<!FULL>(p.w_f32, p.w, col0, p.cols, w);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (E == kWithin) {
            if (const int gone = eight.gone()) raw[i].drop(gone);
        }
        raw[i].get(v[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = FULL || row0 + i < p.rows ? v[i][e] * rstd[i] * w[e] : 0.0f;
    }
    store_tile_columns<NT>(p.q0, tm, tn, FULL ? INT64_MAX : p.cols, v, sh);
}

template <bool SF32, bool NT>
__global__ __launch_bounds__(512) void norm_columns_kernel(NormForward p, Rows h, int tiles_n)
{
    __shared__ TileShared sh;
    const int64_t tm = blockIdx.x / (unsigned)tiles_n, tn = blockIdx.x % (unsigned)tiles_n;
    if ((tm + 1) * 128 <= p.rows && (tn + 1) * 128 <= p.cols)
        norm_tile<SF32, NT, kWhole>(p, h, tm, tn, sh);
    else if (p.cols >= 8)
        norm_tile<SF32, NT, kWithin>(p, h, tm, tn, sh);
    else
        norm_tile<SF32, NT, kFew>(p, h, tm, tn, sh);
}

// Bytes of a call with codes or without.
int64_t forward_bytes(const NormForward &p)
{
    const int x = p.x_f32 ? 4 : 2, s = p.s_f32 ? 4 : 2;
    return p.rows * p.cols * (x + (p.r.p ? s : 0) + (p.h.p ? s : 0) + (p.y.p ? p.y_f32 ? 4 : 2 : 0) + (p.q1.q ? 1 : 0) + (p.q0.q ? 1 : 0));
}

template <bool XF32, bool SF32, bool RES, Ends E, bool NT>
hipError_t pick_forward(const ForwardArgs &args, hipStream_t stream)
{
    const int64_t rows = args.p.rows, cols = args.p.cols, most = (int64_t)1 << 20;
    const auto run = [&](auto kernel, int64_t blocks, int64_t threads) {
        return launch(kernel, dim3((unsigned)std::min(blocks, most)), dim3((unsigned)threads), 0, stream, args);
    };
    if (E == kFew || cols <= 512) return run(norm_forward_kernel<XF32, SF32, RES, E, NT, true, 1>, (rows + 3) / 4, 256);
    if constexpr (E != kFew) {
        if (cols <= 1024) return run(norm_forward_kernel<XF32, SF32, RES, E, NT, true, 2>, (rows + 3) / 4, 256);
        // 16 values a thread: 4096 columns (8192 rows, codes along both axes) 57 us, with 8 values 59, with 32 59, in one wavefront, which
        // needs no barrier, 73
        if (cols <= 16384) return run(norm_forward_kernel<XF32, SF32, RES, E, NT, false, 2>, rows, (cols + 1023) / 1024 * 64);
    }
    return run(norm_forward_long_kernel<XF32, SF32, RES>, rows, 1024);
}
// Streaming loads of x and r and stores of the codes, where the call is more than the last cache takes (outputs in new memory; where rows
// start at multiples of 16 bytes, and where not): 8192 x 4096 in bf16 with codes along both axes (268 MB) 63 -> 60 us and 69 -> 65, 5000 x
// 8192 76 -> 69 and 82 -> 78, 32768 x 1024 61 -> 58 and 61 -> 58, with a bf16 result alone no difference; 4096 x 4096 (134 MB) 32.2 and 32.7.
// With an FP32 stream only for codes along the columns, which read h again (8192 x 8192 207 -> 193 and 212 -> 200; a bf16 result alone
// 153 and 158), and not for x in FP32 (8192 x 4096 109 and 112, with a bf16 result alone 85 and 93). Not for rows that end within eight
// values: 15232 x 5627 202 us, and 212 with them.
template <bool XF32, bool SF32, bool RES>
hipError_t forward(const ForwardArgs &args, bool nt, hipStream_t stream)
{
    const int64_t cols = args.p.cols;
    if (cols % 8)
        return cols < 8 ? pick_forward<XF32, SF32, RES, kFew, false>(args, stream) : pick_forward<XF32, SF32, RES, kWithin, false>(args, stream);
    if constexpr (!XF32) {
        if (nt) return pick_forward<XF32, SF32, RES, kWhole, true>(args, stream);
    }
    return pick_forward<XF32, SF32, RES, kWhole, false>(args, stream);
}

}  // namespace

hipError_t launch_norm_forward(const NormForward &p, hipStream_t stream)
{
    const ForwardArgs args{p, 1.0 / (double)p.cols};
    const bool res = p.r.p != nullptr;
    const bool nt = forward_bytes(p) > kStreamBytes && !p.x_f32 && !(res && p.s_f32 && !p.q0.q);
    hipError_t e;
    if (!res)
        e = p.x_f32 ? forward<true, true, false>(args, nt, stream) : forward<false, false, false>(args, nt, stream);
    else if (p.x_f32)
        e = p.s_f32 ? forward<true, true, true>(args, nt, stream) : forward<true, false, true>(args, nt, stream);
    else
        e = p.s_f32 ? forward<false, true, true>(args, nt, stream) : forward<false, false, true>(args, nt, stream);
    if (e != hipSuccess || !p.q0.q) return e;
    const Rows h = res ? Rows{p.h.p, p.h.ld} : p.x;
    const bool f32 = res ? p.s_f32 : p.x_f32;
    const int64_t tiles_n = (p.cols + 127) / 128;
    const dim3 grid((unsigned)((p.rows + 127) / 128 * tiles_n)), block(512);
    const auto run = [&](auto kernel) { return launch(kernel, grid, block, 0, stream, p, h, (int)tiles_n); };
    if (f32) return run(nt ? norm_columns_kernel<true, true> : norm_columns_kernel<true, false>);
    return run(nt ? norm_columns_kernel<false, true> : norm_columns_kernel<false, false>);
}

}  // namespace mx
