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
// aligned to their elements only. NT: loads and stores that do not stay in the caches, for streams that are larger than those.
template <bool F32>
struct Raw8;
template <>
struct Raw8<false> {
    u32x4 w;
    __device__ __forceinline__ void zero() { w = u32x4{0u, 0u, 0u, 0u}; }
    // what is formed of the values from here on is formed anew, and nothing formed before is kept for it
    __device__ __forceinline__ void renew() { asm volatile("" : "+v"(w)); }
    template <bool NT>
    __device__ __forceinline__ void load(const void *p)
    {
        const u32x4_any *at = reinterpret_cast<const u32x4_any *>(p);
        w = NT ? __builtin_nontemporal_load(at) : *at;
    }
    template <bool NT>
    __device__ __forceinline__ void store(void *p) const
    {
        u32x4_any *at = reinterpret_cast<u32x4_any *>(p);
        if constexpr (NT)
            __builtin_nontemporal_store(w, at);
        else
            *at = w;
    }
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
    // the first n values leave, the others move to their places, zeros behind them
    __device__ __forceinline__ void drop(int n)
    {
        if (n & 4) w = u32x4{w[2], w[3], 0u, 0u};
        if (n & 2) w = u32x4{w[1], w[2], w[3], 0u};
        if (n & 1) w = u32x4{w[0] >> 16 | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | w[3] << 16, w[3] >> 16};
        if (n >= 8) zero();
    }
};
template <>
struct Raw8<true> {
    f32x4 a, b;
    __device__ __forceinline__ void zero() { a = b = f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }
    __device__ __forceinline__ void renew() { asm volatile("" : "+v"(a), "+v"(b)); }
    template <bool NT>
    __device__ __forceinline__ void load(const void *p)
    {
        const f32x4_any *at = reinterpret_cast<const f32x4_any *>(p);
        const f32x4_any *next = reinterpret_cast<const f32x4_any *>(static_cast<const float *>(p) + 4);
        a = NT ? __builtin_nontemporal_load(at) : *at;
        b = NT ? __builtin_nontemporal_load(next) : *next;
    }
    template <bool NT>
    __device__ __forceinline__ void store(void *p) const
    {
        f32x4_any *at = reinterpret_cast<f32x4_any *>(p), *next = reinterpret_cast<f32x4_any *>(static_cast<float *>(p) + 4);
        if constexpr (NT) {
            __builtin_nontemporal_store(a, at);
            __builtin_nontemporal_store(b, next);
        } else {
            *at = a;
            *next = b;
        }
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
    __device__ __forceinline__ void drop(int n)
    {
        if (n & 4) a = b, b = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (n & 2) a = f32x4{a[2], a[3], b[0], b[1]}, b = f32x4{b[2], b[3], 0.0f, 0.0f};
        if (n & 1) a = f32x4{a[1], a[2], a[3], b[0]}, b = f32x4{b[1], b[2], b[3], 0.0f};
        if (n >= 8) zero();
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
template <bool F32, bool RAGGED, bool NT = false>
__device__ __forceinline__ Raw8<F32> load_raw(const void *row, int64_t col, int64_t cols)
{
    Raw8<F32> r;
    if (RAGGED ? col + 8 <= cols : col < cols) {
        r.template load<NT>(at<F32>(row, col));
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
// How a row ends: with whole eights; within eight, but not before the first eight; or before.
enum Ends { kWhole, kWithin, kFew };

// The eight values of a row from col on, for kernels that hold a row in registers. kWithin has no branch around a load (a thread's
// first would be waited for before its second): the row's last eight are read at its end, and those in front of col, gone() of them,
// are dropped once they are there. The norm's gradient of 15000 x 5628 and of 15000 x 5627 takes 160 us so, and 227 and 247
// with load_raw, the forward pass 161 and 195, and 189 and 202; with whole eights, where it takes more registers, 156 and 144.
template <Ends E>
struct Eight {
    int64_t col, cols, from;
    __device__ __forceinline__ Eight(int64_t col, int64_t cols) : col(col), cols(cols), from(E == kWithin ? min(col, cols - 8) : col) {}
    template <bool F32, bool NT>
    __device__ __forceinline__ Raw8<F32> load(const void *row) const
    {
        if constexpr (E != kWithin) return load_raw<F32, E == kFew, NT>(row, col, cols);
        Raw8<F32> r;
        r.template load<NT>(at<F32>(row, from));
        return r;
    }
    // the number of values that are not this thread's, the same for all that it has loaded here
    __device__ __forceinline__ int gone() const { return E == kWithin ? (int)min(col - from, (int64_t)8) : 0; }
};

template <bool F32, bool RAGGED, bool NT = false>
__device__ __forceinline__ void store_raw(const Raw8<F32> &r, void *row, int64_t col, int64_t cols)
{
    if (RAGGED ? col + 8 <= cols : col < cols) {
        r.template store<NT>(at<F32>(row, col));
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
// Bit pattern of the largest of N magnitudes, that of a NaN if one is (v_maximum3_f32 takes two more values at a time and keeps
// NaN, where comparing bit patterns needs the sign off each first).
template <int N>
__device__ __forceinline__ uint32_t largest(const float (&v)[N])
{
    float m = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) m = __builtin_elementwise_maximum(m, fabsf(v[i]));
    return __float_as_uint(m);
}

// Scale bytes that the conversion below does not take: 0 (2^-127, which FP32 does not hold as a normal number) and 0xFF
// (no number). Blocks of zeros, of tiny values, and those that hold a NaN or an infinity.
__device__ __forceinline__ bool special(uint32_t s) { return s - 1u > 253u; }

typedef short i16x2 __attribute__((ext_vector_type(2)));

// Four values over 2^(S - 127), S in [1, 247], as E4M3 codes, rounded to nearest even; the quotient is at most 448. One
// instruction divides and rounds two of them, where encode4 multiplies each first.
__device__ __forceinline__ uint32_t divide4(float a, float b, float c, float d, float scale)
{
    i16x2 w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, scale, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, scale, true);
    return __builtin_bit_cast(uint32_t, w);
}
// The same with any S: codes 0 for 0xFF.
__device__ __forceinline__ uint32_t divide4_any(float a, float b, float c, float d, uint32_t s)
{
    return s == 0xFFu ? 0u : encode4(a, b, c, d, inverse_scale(s));
}

// Eight values of a row in each of 16 lanes side by side, which are one block: their codes, and the block's scale byte.
__device__ __forceinline__ u32x2 row_codes(const float (&v)[8], uint32_t &s)
{
    s = e8m0_of(row16_max(largest(v)) & 0x7FFFFFFFu);
    if (__any(special(s))) return u32x2{divide4_any(v[0], v[1], v[2], v[3], s), divide4_any(v[4], v[5], v[6], v[7], s)};
    const float scale = __uint_as_float(s << 23);
    return u32x2{divide4(v[0], v[1], v[2], v[3], scale), divide4(v[4], v[5], v[6], v[7], scale)};
}
template <bool NT>
__device__ __forceinline__ void store_codes(const u32x2 &w, uint8_t *to)
{
    if constexpr (NT)
        __builtin_nontemporal_store(w, reinterpret_cast<u32x2 *>(to));
    else
        *reinterpret_cast<u32x2 *>(to) = w;
}
// The same, written: col a multiple of 8, the block's first lane at a multiple of 128; zeros behind the row's end up to the
// block's.
template <bool NT>
__device__ __forceinline__ void store_row_codes(const Fp8Out &out, int64_t row, int64_t col, int64_t cols, const float (&v)[8])
{
    uint32_t s;
    const u32x2 w = row_codes(v, s);
    if ((col & ~(int64_t)127) >= cols) return;
    store_codes<NT>(w, out.q + row * out.ldq + col);
    if ((col & 127) == 0) out.s[row * out.lds + (col >> 7)] = (uint8_t)s;
}

// A tile of 128 x 128 values in 512 threads of 4 x 8: thread t has rows 4 (t / 16) .. and columns 8 (t % 16) .. .
// Along the columns a block is a column of the tile: its maximum joins the four row groups of a wavefront by
// lane swaps and the wavefronts through the LDS, which also turns the codes.
// Workgroups go round the eight XCDs one by one: each XCD takes a run of tiles side by side (gated activation 8192 x 14336 125 ->
// 121 us, its gradient 260 -> 243; the norm's codes along the columns, whose input is in the caches, in their own order).
struct Tile {
    int64_t m, n;
};
__device__ __forceinline__ Tile tile_of(int tiles_n)
{
    const unsigned each = gridDim.x / 8, b = blockIdx.x, id = b < 8 * each ? b % 8 * each + b / 8 : b;
    return {id / (unsigned)tiles_n, id % (unsigned)tiles_n};
}

struct TileShared {
    uint32_t top[8][128];
    uint32_t scale[128];      // scale bytes as FP32's exponents
    uint32_t special[2];
    // a column's 128 codes, in 16-byte chunks permuted by the column's bits 3-5 against bank conflicts
    __attribute__((aligned(16))) uint8_t turned[128 * 128];
};

// tm, tn: the tile's place. Values behind the matrix' ends are zeros. Every thread of the workgroup calls it, and may do so
// again at once: what a call still reads behind its last barrier, the next one writes behind its first.
template <bool NT>
__device__ __forceinline__ void store_tile_columns(const Fp8Out &out, int64_t tm, int64_t tn, int64_t cols,
                                                   const float (&v)[4][8], TileShared &sh)
{
    const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
    uint32_t m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float column[4] = {v[0][j], v[1][j], v[2][j], v[3][j]};
        m[j] = largest(column);
    }
    // Lanes 16 further have the next four rows of the same columns. A swap of the odd groups of 16 lanes of one register with
    // the even ones of another leaves both groups' maxima of one column beside each other, and another column's in the other
    // group; so does one of the wavefront's halves. A lane ends with two columns' maxima over 16 rows.
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const auto r = __builtin_amdgcn_permlane16_swap(m[j], m[j + 4], false, false);
        m[j] = max(r[0], r[1]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const auto r = __builtin_amdgcn_permlane32_swap(m[j], m[j + 2], false, false);
        m[j] = max(r[0], r[1]);
    }
    *reinterpret_cast<u32x2 *>(&sh.top[tid >> 6][8 * cg + 4 * (rg & 1) + (rg & 2)]) = u32x2{m[0], m[1]};
    __syncthreads();
    if (tid < 128) {
        uint32_t top = sh.top[0][tid];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = max(top, sh.top[i][tid]);
        const uint32_t s = e8m0_of(top & 0x7FFFFFFFu);
        sh.scale[tid] = s << 23;
        const bool any = __any(special(s));
        if ((tid & 63) == 0) sh.special[tid >> 6] = any ? 1u : 0u;
    }
    __syncthreads();
    // four codes from row 4 rg on: bytes 4 (rg % 4) of chunk rg / 4 of the column
    uint8_t *to = sh.turned + 8 * cg * 128 + 16 * ((rg >> 2) ^ (cg & 7)) + 4 * (rg & 3);
    const u32x4 s0 = *reinterpret_cast<const u32x4 *>(sh.scale + 8 * cg), s1 = *reinterpret_cast<const u32x4 *>(sh.scale + 8 * cg + 4);
    const bool slow = (sh.special[0] | sh.special[1]) != 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t s = j < 4 ? s0[j & 3] : s1[j & 3];
        *reinterpret_cast<uint32_t *>(to + j * 128) = slow ? divide4_any(v[0][j], v[1][j], v[2][j], v[3][j], s >> 23)
                                                           : divide4(v[0][j], v[1][j], v[2][j], v[3][j], __uint_as_float(s));
    }
    __syncthreads();
    // eight lanes write a column's 128 bytes
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int col = 64 * p + (tid >> 3), chunk = tid & 7;
        const int64_t outer = tn * 128 + col;
        if (outer >= cols) continue;
        const u32x4 w = *reinterpret_cast<const u32x4 *>(sh.turned + col * 128 + 16 * (chunk ^ ((col >> 3) & 7)));
        u32x4 *to = reinterpret_cast<u32x4 *>(out.q + outer * out.ldq + tm * 128 + 16 * chunk);
        if constexpr (NT)
            __builtin_nontemporal_store(w, to);
        else
            *to = w;
        if (chunk == 0) out.s[outer * out.lds + tm] = (uint8_t)(sh.scale[col] >> 23);
    }
}

}  // namespace mx
