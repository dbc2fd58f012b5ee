// Device-side building blocks of the operators between the products: eight values of a row at a time, sums over
// lanes, and 8-bit outputs of rows and of 128 x 128 tiles.
#pragma once

#include "fp8_device.h"
#include "layer_internal.h"

namespace mx {

typedef __bf16 bf16_pair_t __attribute__((ext_vector_type(2)));

// two values as bf16, rounded to nearest even
__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const bf16_pair_t v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// -------------------------------------------------------------------- eight values of a row ---
// As they lie in memory, so that a thread's loads can all be under way before the first is used. Rows are
// aligned to their elements only.
template <bool F32>
struct Raw8;
template <>
struct Raw8<false> {
    u32x4 w;
    __device__ __forceinline__ void zero() { w = u32x4{0u, 0u, 0u, 0u}; }
    __device__ __forceinline__ void load(const void *p)
    {
        w = *reinterpret_cast<const u32x4_any *>(p);
    }
    __device__ __forceinline__ void store(void *p) const { *reinterpret_cast<u32x4_any *>(p) = w; }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = bf16_lo(w[e]);
            v[2 * e + 1] = bf16_hi(w[e]);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8])
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = bf16_pair(v[2 * e], v[2 * e + 1]);
    }
};
template <>
struct Raw8<true> {
    f32x4 a, b;
    __device__ __forceinline__ void zero() { a = b = f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }
    __device__ __forceinline__ void load(const void *p)
    {
        a = *reinterpret_cast<const f32x4_any *>(p);
        b = *reinterpret_cast<const f32x4_any *>(static_cast<const float *>(p) + 4);
    }
    __device__ __forceinline__ void store(void *p) const
    {
        *reinterpret_cast<f32x4_any *>(p) = a;
        *reinterpret_cast<f32x4_any *>(static_cast<float *>(p) + 4) = b;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = a[e];
            v[4 + e] = b[e];
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8])
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            a[e] = v[e];
            b[e] = v[4 + e];
        }
    }
};

template <bool F32>
__device__ __forceinline__ const void *at(const void *p, int64_t i)
{
    return static_cast<const char *>(p) + i * (F32 ? 4 : 2);
}
template <bool F32>
__device__ __forceinline__ void *at(void *p, int64_t i)
{
    return static_cast<char *>(p) + i * (F32 ? 4 : 2);
}

// Values col .. col + 7 of a row that starts at `row` and has `cols`; zeros behind its end. RAGGED: it may end within
// these eight (they are then read one by one); otherwise col and cols are multiples of eight.
template <bool F32, bool RAGGED>
__device__ __forceinline__ Raw8<F32> load_raw(const void *row, int64_t col, int64_t cols)
{
    Raw8<F32> r;
    if (RAGGED ? col + 8 <= cols : col < cols) {
        r.load(at<F32>(row, col));
        return r;
    }
    r.zero();
    if constexpr (RAGGED) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (col + e >= cols) break;
            if constexpr (F32) {
                const float x = static_cast<const float *>(row)[col + e];
                if (e < 4)
                    r.a[e & 3] = x;
                else
                    r.b[e & 3] = x;
            } else {
                r.w[e / 2] |= (uint32_t)static_cast<const uint16_t *>(row)[col + e] << (16 * (e & 1));
            }
        }
    }
    return r;
}
template <bool F32, bool RAGGED>
__device__ __forceinline__ void store_raw(const Raw8<F32> &r, void *row, int64_t col, int64_t cols)
{
    if (RAGGED ? col + 8 <= cols : col < cols) {
        r.store(at<F32>(row, col));
        return;
    }
    if constexpr (RAGGED) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (col + e >= cols) break;
            if constexpr (F32)
                static_cast<float *>(row)[col + e] = e < 4 ? r.a[e & 3] : r.b[e & 3];
            else
                static_cast<uint16_t *>(row)[col + e] = (uint16_t)(r.w[e / 2] >> (16 * (e & 1)));
        }
    }
}
// the same with the type known at run time only (the same for all lanes)
template <bool RAGGED>
__device__ __forceinline__ void load_any(bool f32, const void *row, int64_t col, int64_t cols, float (&v)[8])
{
    if (f32)
        load_raw<true, RAGGED>(row, col, cols).get(v);
    else
        load_raw<false, RAGGED>(row, col, cols).get(v);
}
template <bool RAGGED>
__device__ __forceinline__ void store_any(bool f32, const float (&v)[8], void *row, int64_t col, int64_t cols)
{
    if (f32) {
        Raw8<true> r;
        r.set(v);
        store_raw<true, RAGGED>(r, row, col, cols);
    } else {
        Raw8<false> r;
        r.set(v);
        store_raw<false, RAGGED>(r, row, col, cols);
    }
}

// ------------------------------------------------------------------------- sums over lanes ----
template <class T>
__device__ __forceinline__ T wave_sum(T v)
{
#pragma unroll
    for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

// ---------------------------------------------------------------------------- 8-bit outputs ---
// Eight values of a row in each of 16 lanes side by side, which are one block (col a multiple of 8, the block's
// first lane at a multiple of 128): its codes, zeros behind the row's end up to the block's, and its scale.
__device__ __forceinline__ void store_row_codes(const Fp8Out &out, int64_t row, int64_t col, int64_t cols, const float (&v)[8])
{
    const uint32_t s = e8m0_of(row16_max(amax_bits<8>(v)));
    const float inv = inverse_scale(s == 0xFFu ? 0u : s);
    u32x2 w = {0u, 0u};
    if (s != 0xFFu) w = u32x2{encode4(v[0], v[1], v[2], v[3], inv), encode4(v[4], v[5], v[6], v[7], inv)};
    if ((col & ~(int64_t)127) >= cols) return;
    *reinterpret_cast<u32x2 *>(out.q + row * out.ldq + col) = w;
    if ((col & 127) == 0) out.s[row * out.lds + (col >> 7)] = (uint8_t)s;
}

// A tile of 128 x 128 values in 16 * 128 / N threads of N x 8: thread t has rows N (t / 16) .. and columns
// 8 (t % 16) .. . Along the columns a block is a column of the tile: its maximum joins the four row groups of
// a wavefront by lane swaps and the wavefronts through the LDS, which also turns the codes.
template <int N>
struct TileShared {
    static constexpr int kWaves = 16 * 128 / N / 64;
    uint32_t cmax[kWaves][128];
    uint32_t scale[128];
    // a column's 128 codes, in 16-byte chunks permuted by the column's bits 3-5 against bank conflicts
    __attribute__((aligned(16))) uint8_t turned[128 * 128];
};

__device__ __forceinline__ uint32_t rows_max(uint32_t v)
{
    auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(r[0], r[1]);
    r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max(r[0], r[1]);
}

// tm, tn: the tile's place. Values behind the matrix' ends are zeros. Every thread of the workgroup calls it; `sh` may be
// used again after the next barrier.
template <int N>
__device__ __forceinline__ void store_tile_columns(const Fp8Out &out, int64_t tm, int64_t tn, int64_t cols,
                                                   const float (&v)[N][8], TileShared<N> &sh)
{
    constexpr int kThreads = 16 * 128 / N;
    const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
    uint32_t m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        m[j] = 0u;
#pragma unroll
        for (int i = 0; i < N; ++i) m[j] = max(m[j], abs_bits(v[i][j]));
        m[j] = rows_max(m[j]);
    }
    if ((tid & 48) == 0) {
        u32x4 *to = reinterpret_cast<u32x4 *>(&sh.cmax[tid >> 6][8 * cg]);
        to[0] = u32x4{m[0], m[1], m[2], m[3]};
        to[1] = u32x4{m[4], m[5], m[6], m[7]};
    }
    __syncthreads();
    if (tid < 128) {
        uint32_t top = sh.cmax[0][tid];
#pragma unroll
        for (int i = 1; i < TileShared<N>::kWaves; ++i) top = max(top, sh.cmax[i][tid]);
        sh.scale[tid] = e8m0_of(top);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int col = 8 * cg + j;
        const uint32_t s = sh.scale[col];
        const float inv = inverse_scale(s == 0xFFu ? 0u : s);
        // N codes from row N rg on: chunk (N rg) / 16 of the column
        uint8_t *to = sh.turned + col * 128 + 16 * (((N * rg) >> 4) ^ (cg & 7)) + ((N * rg) & 15);
        if constexpr (N == 8)
            *reinterpret_cast<u32x2 *>(to) = s == 0xFFu ? u32x2{0u, 0u}
                                                        : u32x2{encode4(v[0][j], v[1][j], v[2][j], v[3][j], inv),
                                                                encode4(v[4][j], v[5][j], v[6][j], v[7][j], inv)};
        else
            *reinterpret_cast<uint32_t *>(to) = s == 0xFFu ? 0u : encode4(v[0][j], v[1][j], v[2][j], v[3][j], inv);
    }
    __syncthreads();
    // eight lanes write a column's 128 bytes
#pragma unroll
    for (int p = 0; p < 1024 / kThreads; ++p) {
        const int col = (kThreads / 8) * p + (tid >> 3), chunk = tid & 7;
        const int64_t outer = tn * 128 + col;
        if (outer >= cols) continue;
        *reinterpret_cast<u32x4 *>(out.q + outer * out.ldq + tm * 128 + 16 * chunk) =
            *reinterpret_cast<const u32x4 *>(sh.turned + col * 128 + 16 * (chunk ^ ((col >> 3) & 7)));
        if (chunk == 0) out.s[outer * out.lds + tm] = (uint8_t)sh.scale[col];
    }
}

}  // namespace mx
