// Newton-Schulz orthogonalisation of a matrix (or a batch of one shape):
//
//   X = G / (|G|_F + eps);  steps times:  A = X X^T,  X <- a X + (b A + c A A) X;  out = alpha X + beta out
//
// with the Gram matrix taken along the shorter side (X^T X for more rows than columns). The
// products run on the FP16 matrix cores with FP32 accumulation. FP16 holds 2^10 X, 2^10 A and
// 2^10 (b A + c A A): every entry of X stays below 1.3 and of the others below 3 in magnitude
// (singular values of X lie in [0, 1.3] at every step for the usual coefficients), so nothing
// overflows (other coefficients are checked on the host to stay within FP16, t below is held to 16), and
// entries down to 2^-24 keep all 11 bits. X itself is carried from step to step in two FP16
// numbers, value and remainder (22 bits): the term a X, which carries the small singular values,
// loses nothing, and what the 11-bit operands add stays below the rounding of a bf16 result
// (with X in FP16 alone a matrix of a few strong directions was off by 0.011, with bf16 operands by 0.09).
//
// Near singular values of 1 the two terms of the update nearly cancel, and the roundings of b A + c A A and
// of the X that it is multiplied by count |b + c| times (2.7). A step may as well be (a - t) X +
// (b A + c A A + t) X: with t = -(b + c) they count next to nothing there, but t times for the directions that
// are still small, and what those pick up grows with them in the steps that follow. So the last step takes
// t = -(b + c), the one before it a half of it, and the others none. Relative error in five steps,
// sides of 65 to 2048: heavy tails 0.0008 to 0.0017, without t 0.0012 to 0.0020; one strong direction over noise of 1/10
// 0.0004, of 1/1000 0.0014, of less 0.0016 to 0.0018 (without t 0.0002 to 0.0007: the noise's directions then hold little but
// these roundings). A quarter of t in the third last step as well: 0.0008 to 0.0014, but 0.0032 over little noise; t in every
// step 0.03. A bf16 result's own rounding is 0.0017. Matrices with a side of at most 64 are worked in FP32 (below).
//
// Per step three launches: A (symmetric: the lower triangle of tiles, written twice), b A + c A A
// (symmetric too), and the update, which writes X in both orientations for the next step's
// products, each of which contracts along rows.
//
// Bound by the matrix cores: 4096 x 4096 in 1.45 ms, of which the four updates 121 us each (1.14 PFLOP/s; they write X
// three times), the last one 110, and the ten symmetric products 82 each, whose 136 tiles leave 120 CUs idle (in 128 x 128
// tiles, which fill them, they take longer); norm and first operands 32. 14336 x 4096: 4.09 ms; an update 429 us + 27 for the
// half round of its 896 tiles that is split, the last 386 + 20, A 226 + 26, b A + c A A 89, norm and first operands 151. 2 x
// 1024 x 4096: 0.32 ms; 22, 9 and 30 us a step. Small ones by each launch's own latency: 256 x 512 takes 79 us in 17, each 4
// to 6 us. (Kernels and wholes from one session, 60 calls on end.)
#include <algorithm>

#include "slab_gemm.h"
#include "train_internal.h"

namespace mx {
namespace {

using namespace slab;

constexpr float kUnscale = 1.0f / 1024.0f;
constexpr float kLoScale = 2048.0f, kLoUnscale = 1.0f / 2048.0f;   // the remainder, held 2^11 larger

__device__ __forceinline__ uint16_t f16_bits(float x) { return __builtin_bit_cast(uint16_t, (_Float16)x); }
__device__ __forceinline__ float f16_float(uint16_t b) { return (float)__builtin_bit_cast(_Float16, b); }
// eight FP16 values
__device__ __forceinline__ void f16_eight(const u32x4 &w, f32x4 (&v)[2])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t word = w[k];   // copied out first: a bit cast of a vector's element reads the vector's first one
        const f16x2 two = __builtin_bit_cast(f16x2, word);
        v[k / 2][2 * (k % 2)] = (float)two[0];
        v[k / 2][2 * (k % 2) + 1] = (float)two[1];
    }
}

// ------------------------------------------------------------------------- the epilogues ------
// A = X X^T: 2^20 A in acc, 2^10 A stored, in both places
struct GramEpi {
    static constexpr bool kSym = true;
    uint16_t *out;
    int64_t ld, batch_out;
    template <class G>
    __device__ __forceinline__ void run(f32x4 (&acc)[G::FI][G::FJ], const Where &w, const Operands &, uint8_t *lds,
                                        uint8_t *) const
    {
        uint16_t *o = out + w.batch * batch_out;
        store_tile16<G>(acc, w, lds, [](float a, float b) { return pack_f16(a, b); }, [](int, int) { return 0; },
                        [&](f32x4 (&v)[2], int, int, int) {
                            v[0] *= kUnscale;
                            v[1] *= kUnscale;
                        },
                        o, ld, w.m0 == w.n0 ? nullptr : o, ld);
    }
};

// b A + c A A + t: 2^20 A A in acc, 2^10 A read
struct PolyEpi {
    static constexpr bool kSym = true;
    const uint16_t *gram;
    uint16_t *out;
    int64_t ld, batch_out;
    float b, c, t;
    template <class G>
    __device__ __forceinline__ void run(f32x4 (&acc)[G::FI][G::FJ], const Where &w, const Operands &, uint8_t *lds,
                                        uint8_t *) const
    {
        const uint16_t *in = gram + w.batch * batch_out;
        uint16_t *o = out + w.batch * batch_out;
        const float cs = c * kUnscale;
        store_tile16<G>(acc, w, lds, [](float x, float y) { return pack_f16(x, y); },
                        [&](int m, int n) { return *reinterpret_cast<const u32x4 *>(in + (int64_t)m * ld + n); },
                        [&](f32x4 (&v)[2], const u32x4 &gram8, int m, int n) {
                            f32x4 g[2];
                            f16_eight(gram8, g);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                v[k] = b * g[k] + cs * v[k];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (m == n + 4 * k + e) v[k][e] += 1024.0f * t;
                            }
                        },
                        o, ld, w.m0 == w.n0 ? nullptr : o, ld);
    }
};

// eight values of X as they are kept
struct TwoPart {
    u32x4 hi, lo;
    __device__ __forceinline__ void read(f32x4 (&x)[2]) const
    {
        f32x4 rest[2];
        f16_eight(hi, x);
        f16_eight(lo, rest);
        x[0] += rest[0] * kLoUnscale;
        x[1] += rest[1] * kLoUnscale;
    }
};
__device__ __forceinline__ TwoPart two_part(const uint16_t *hi, const uint16_t *lo, int64_t at)
{
    return TwoPart{*reinterpret_cast<const u32x4 *>(hi + at), *reinterpret_cast<const u32x4 *>(lo + at)};
}

// (a - t) X + (b A + c A A + t) X in X's own orientation: value (both orientations) and remainder
struct UpdateEpi {
    static constexpr bool kSym = false;
    const uint16_t *hi;      // X [mp][np]
    uint16_t *lo;            // read and written
    uint16_t *hi_out, *turned_out;
    int64_t ld, ld_turned, batch_x;
    float a;
    template <class G>
    __device__ __forceinline__ void run(f32x4 (&acc)[G::FI][G::FJ], const Where &w, const Operands &, uint8_t *lds,
                                        uint8_t *) const
    {
        const int64_t base = w.batch * batch_x;
        store_tile16<G>(acc, w, lds, [](float x, float y) { return pack_f16(x, y); },
                        [&](int m, int n) { return two_part(hi, lo, base + (int64_t)m * ld + n); },
                        [&](f32x4 (&v)[2], const TwoPart &two, int m, int n) {
                            f32x4 x[2];
                            two.read(x);
                            u32x4 rests;
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                v[k] = a * x[k] + kUnscale * v[k];
                                float rest[4];
#pragma unroll
                                for (int t = 0; t < 4; ++t) rest[t] = (v[k][t] - f16_float(f16_bits(v[k][t]))) * kLoScale;
                                rests[2 * k] = pack_f16(rest[0], rest[1]);
                                rests[2 * k + 1] = pack_f16(rest[2], rest[3]);
                            }
                            *reinterpret_cast<u32x4 *>(lo + base + (int64_t)m * ld + n) = rests;
                        },
                        hi_out + base, ld, turned_out + base, ld_turned);
    }
};

// the last update, straight into the caller's matrix: out = alpha X + beta out
template <bool BF16_OUT>
struct LastEpi {
    static constexpr bool kSym = false;
    const uint16_t *hi, *lo;
    int64_t ld, batch_x;
    float a;
    StoreEpi<BF16_OUT> store;   // alpha covers X's 2^10
    template <class G>
    __device__ __forceinline__ void run(f32x4 (&acc)[G::FI][G::FJ], const Where &w, const Operands &op, uint8_t *lds,
                                        uint8_t *) const
    {
        const int64_t base = w.batch * batch_x;
        store.template run_with<G>(acc, w, op, lds, [&](int m, int n) { return two_part(hi, lo, base + (int64_t)m * ld + n); },
                                   [&](f32x4 (&v)[2], const TwoPart &two) {
                                       f32x4 x[2];
                                       two.read(x);
                                       v[0] = a * x[0] + kUnscale * v[0];
                                       v[1] = a * x[1] + kUnscale * v[1];
                                   });
    }
};

// ----------------------------------------------------------------- norm and first operands ----
constexpr int kNormBlocks = 1024;   // at most so many partial sums of a matrix
constexpr int kNormTile = 8192;     // values a workgroup should at least have

template <bool F32>
__device__ __forceinline__ float read_g(const void *g, int64_t at)
{
    if constexpr (F32)
        return static_cast<const float *>(g)[at];
    else
        return bf16_float(static_cast<const uint16_t *>(g)[at]);
}

// eight consecutive values; 16-byte aligned
template <bool F32>
__device__ __forceinline__ void read_g8(const void *g, int64_t at, float (&v)[8])
{
    if constexpr (F32) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(g) + at);
        const f32x4 b = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(g) + at + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = a[e];
            v[4 + e] = b[e];
        }
    } else {
        const u32x4 a = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(g) + at);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t word = a[e];
            v[2 * e] = bf16_float(word & 0xFFFFu);
            v[2 * e + 1] = bf16_float(word >> 16);
        }
    }
}

// Sums of squares, one per workgroup, in 64 bits (the squares of FP32 numbers leave FP32's range). Bound by
// memory: 14336 x 4096 in FP32 52 us, 4.5 TB/s. vec: 16-byte aligned rows of whole eights.
template <bool F32>
__global__ __launch_bounds__(256) void norm_kernel(const void *__restrict__ g, int64_t m, int64_t n, int64_t ldg, int64_t batch_g,
                                                   int vec, double *__restrict__ part)
{
    __shared__ double slots[4];
    const int64_t base = blockIdx.z * batch_g;
    double sum = 0.0;
    if (vec) {
        const int64_t per_row = n / 8;
        // a thread's eights of its row run on by 256; rows of fewer than that share the workgroup
        const int64_t across = per_row < 256 ? per_row : 256, rows_at_once = 256 / across;
        const int64_t lane_row = threadIdx.x / across, lane_col = threadIdx.x % across;
        if (lane_row < rows_at_once)
            for (int64_t row = blockIdx.x * rows_at_once + lane_row; row < m; row += (int64_t)gridDim.x * rows_at_once)
                for (int64_t c = lane_col; c < per_row; c += across) {
                    float v[8];
                    read_g8<F32>(g, base + row * ldg + 8 * c, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum += (double)v[e] * (double)v[e];
                }
    } else {
        for (int64_t row = blockIdx.x; row < m; row += gridDim.x)
            for (int64_t col = threadIdx.x; col < n; col += 256) {
                const double v = (double)read_g<F32>(g, base + row * ldg + col);
                sum += v * v;
            }
    }
    for (int k = 32; k >= 1; k >>= 1) sum += __shfl_xor(sum, k);
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) part[blockIdx.z * kNormBlocks + blockIdx.x] = (slots[0] + slots[1]) + (slots[2] + slots[3]);
}

// `times` / (|G| + eps), from the partial sums of blockIdx.z's matrix: 2^-power times the result (the factor may lie outside
// FP32's range where G's entries do not). By every workgroup of 256 threads, with a barrier.
__device__ __forceinline__ float norm_factor(const double *part, int parts, float eps, double times, int &power)
{
    __shared__ double slots[4];
    double sum = 0.0;
    for (int k = threadIdx.x; k < parts; k += 256) sum += part[blockIdx.z * kNormBlocks + k];
    for (int k = 32; k >= 1; k >>= 1) sum += __shfl_xor(sum, k);
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = sum;
    __syncthreads();
    const double norm = sqrt((slots[0] + slots[1]) + (slots[2] + slots[3])) + (double)eps;
    power = norm > 0.0 && norm <= 1e300 ? ilogb(norm) : 0;
    return (float)(times / ldexp(norm, -power));
}

// X = G / (|G| + eps), times 2^10, in value and remainder and (the value) transposed, with zeros around it.
// 128 x 128 tiles: a thread takes 8 x 8 values and transposes them in registers; 256-byte lines of
// the transposed are put together in the LDS. Bound by memory: 4 (or 2) bytes in, 6 out; 14336 x 4096 from FP32
// 99 us (5.9 TB/s, some of it from the cache that the norm's read has filled).
template <bool F32>
__global__ __launch_bounds__(256) void first_kernel(const void *__restrict__ g, int64_t m, int64_t n, int64_t ldg, int64_t batch_g,
                                                    int vec, const double *__restrict__ part, int parts, float eps,
                                                    uint16_t *__restrict__ hi, uint16_t *__restrict__ lo,
                                                    uint16_t *__restrict__ turned, int64_t mp, int64_t np, int64_t batch_x)
{
    __shared__ __attribute__((aligned(16))) uint16_t tile[128 * 128];   // [column][row], 16-byte pieces permuted
    int power;
    const float inv = norm_factor(part, parts, eps, 1024.0, power);

    const int64_t r0 = (int64_t)blockIdx.x * 128, c0 = (int64_t)blockIdx.y * 128;
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int64_t c = c0 + 8 * cg;
    uint16_t h[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 8 * rg + i, at = blockIdx.z * batch_g + r * ldg + c;
        float v[8];
        if (vec && r < m && c + 8 <= n) {
            read_g8<F32>(g, at, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = r < m && c + e < n ? read_g<F32>(g, at + e) : 0.0f;
        }
        u32x4 value, rest;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a = ldexpf(v[2 * e], -power) * inv, b = ldexpf(v[2 * e + 1], -power) * inv;
            h[i][2 * e] = f16_bits(a);
            h[i][2 * e + 1] = f16_bits(b);
            value[e] = (uint32_t)h[i][2 * e] | (uint32_t)h[i][2 * e + 1] << 16;
            rest[e] = pack_f16((a - f16_float(h[i][2 * e])) * kLoScale, (b - f16_float(h[i][2 * e + 1])) * kLoScale);
        }
        *reinterpret_cast<u32x4 *>(hi + blockIdx.z * batch_x + r * np + c) = value;
        *reinterpret_cast<u32x4 *>(lo + blockIdx.z * batch_x + r * np + c) = rest;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        u32x4 o;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = (uint32_t)h[2 * k][e] | (uint32_t)h[2 * k + 1][e] << 16;
        *reinterpret_cast<u32x4 *>(tile + (8 * cg + e) * 128 + 8 * (rg ^ cg)) = o;
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int col = 16 * p + (threadIdx.x >> 4), piece = threadIdx.x & 15;
        *reinterpret_cast<u32x4 *>(turned + blockIdx.z * batch_x + (c0 + col) * mp + r0 + 8 * piece) =
            *reinterpret_cast<const u32x4 *>(tile + col * 128 + 8 * (piece ^ (col >> 3)));
    }
}

// out[at] = v + beta out[at], which is read only when beta != 0
__device__ __forceinline__ void put_out(void *out, int bf16, int64_t at, float v, float beta)
{
    if (bf16) {
        uint16_t *p = static_cast<uint16_t *>(out) + at;
        if (beta != 0.0f) v += beta * bf16_float(*p);
        *p = (uint16_t)(pack_bf16(v, 0.0f) & 0xFFFFu);
    } else {
        float *p = static_cast<float *>(out) + at;
        if (beta != 0.0f) v += beta * *p;
        *p = v;
    }
}

// steps == 0: out = alpha X + beta out from the first operands
__global__ __launch_bounds__(256) void copy_out_kernel(const uint16_t *__restrict__ hi, const uint16_t *__restrict__ lo, int64_t np,
                                                       int64_t batch_x, int64_t m, int64_t n, float alpha, float beta, void *out,
                                                       int bf16, int64_t ldo, int64_t batch_o)
{
    const int64_t total = m * n;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / n, c = i % n, at = blockIdx.z * batch_x + r * np + c, o = blockIdx.z * batch_o + r * ldo + c;
        put_out(out, bf16, o, alpha * ((f16_float(hi[at]) + f16_float(lo[at]) * kLoUnscale) * kUnscale), beta);
    }
}

// ----------------------------------------------------------------------------- thin matrices --
// A short side of at most 64: FP32 throughout, on the FP32 matrix cores. The few roundings of FP16 operands do not average
// out here (an error of 0.0012 to 0.0037, below 16 now and then 0.01; so 1e-6 to 7e-5), and the work is little. Y, X with its
// long side down, is [lp][64]; a step is one kernel: every workgroup forms Q = a + b A + c A A for itself, turns its rows of Y
// into Y Q in place, and adds up their part of the next A. With more than kThinFew parts thin_sum_kernel adds them up in
// between.
// Bound by each launch's own latency: in us, with FP16 operands in 128 x 128 padding and so: 16 x 16 67 and 44; 20 x 10368 120
// and 76; 64 x 14336 130 and 82; 8 of 16 x 14336 553 and 205; 1024 of 64 x 64 1712 and 120. (65 x 4096 in FP16: 101.)
constexpr int kThin = 64, kThinTile = kThin * kThin;
constexpr int kThinLine = kThin + 4;   // floats from a row to the next in the LDS: 16 rows of 4 values meet 64 distinct banks
constexpr int kThinChunks = 256;       // workgroups a matrix is worked by, at most
constexpr int kThinFew = 8;

struct Thin {
    const void *g;
    int f32, bf16, wide;        // G's type, out's type; wide: the short side runs down G
    int64_t s, l, ldg, batch_g; // the short and the long side
    const double *norms;
    int norm_parts;
    float eps;
    float *y;
    int64_t lp;
    int blocks;                 // of 64 rows, for each workgroup
    const float *gram;          // [batch][parts][64][64]
    int parts;
    float *gram_out;            // [batch][gridDim.x][64][64]
    float a, b, c, alpha, beta;
    void *out;
    int64_t ldo, batch_o;
};

// acc[j], 16 rows from `rows` against 16 j .. of `cols`, over 64 values along both their rows; element t: row 4 (lane / 16) + t,
// column 16 j + lane % 16
__device__ __forceinline__ void thin_product(const float *rows, const float *cols, int lane, f32x4 (&acc)[4])
{
    const int at = (lane & 15) * kThinLine + (lane >> 4);
#pragma unroll 4
    for (int k = 0; k < kThin; k += 4) {
        const float x = rows[at + k];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x, cols[at + 16 * j * kThinLine + k], acc[j], 0, 0, 0);
    }
}

// FIRST: from G, scaled to norm 1, instead of a step. LAST: into the caller's matrix.
template <bool FIRST, bool LAST>
__global__ __launch_bounds__(256) void thin_kernel(Thin p)
{
    __shared__ __attribute__((aligned(16))) float q[kThin * kThinLine], y[kThin * kThinLine];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, low = lane >> 4;
    const int64_t z = blockIdx.z;
    int power = 0;
    float inv = 0.0f;
    if constexpr (FIRST) {
        inv = norm_factor(p.norms, p.norm_parts, p.eps, 1.0, power);
    } else {
        const float *gram = p.gram + z * p.parts * kThinTile;
        for (int e = 4 * tid; e < kThinTile; e += 1024) {
            f32x4 v = *reinterpret_cast<const f32x4 *>(gram + e);
            for (int k = 1; k < p.parts; ++k) v += *reinterpret_cast<const f32x4 *>(gram + k * kThinTile + e);
            *reinterpret_cast<f32x4 *>(y + e / kThin * kThinLine + e % kThin) = v;
        }
        __syncthreads();
        // A is symmetric to the bit (both places add the same products in one order), and so is Q
        f32x4 acc[4] = {};
        thin_product(y + 16 * wave * kThinLine, y, lane, acc);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int i = 16 * wave + 4 * low + t, col = 16 * j + r, at = i * kThinLine + col;
                const float v = p.b * y[at] + p.c * acc[j][t];
                q[at] = i == col ? v + p.a : v;
            }
        __syncthreads();
    }
    f32x4 sum[4] = {};
    for (int k = 0; k < p.blocks; ++k) {
        const int64_t row0 = ((int64_t)blockIdx.x * p.blocks + k) * kThin;
        if (row0 >= p.lp) break;
        float *rows = p.y + (z * p.lp + row0) * kThin;
        if constexpr (FIRST) {
            for (int e = tid; e < kThinTile; e += 256) {
                // neighbouring threads along G's rows
                const int i = p.wide ? e % kThin : e / kThin, j = p.wide ? e / kThin : e % kThin;
                float v = 0.0f;
                if (row0 + i < p.l && j < p.s) {
                    const int64_t at = z * p.batch_g + (p.wide ? j * p.ldg + row0 + i : (row0 + i) * p.ldg + j);
                    v = p.f32 ? read_g<true>(p.g, at) : read_g<false>(p.g, at);
                }
                y[i * kThinLine + j] = ldexpf(v, -power) * inv;
            }
            __syncthreads();
        } else {
            for (int e = 4 * tid; e < kThinTile; e += 1024)
                *reinterpret_cast<f32x4 *>(y + e / kThin * kThinLine + e % kThin) = *reinterpret_cast<const f32x4 *>(rows + e);
            __syncthreads();
            f32x4 acc[4] = {};
            thin_product(y + 16 * wave * kThinLine, q, lane, acc);
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int t = 0; t < 4; ++t) y[(16 * wave + 4 * low + t) * kThinLine + 16 * j + r] = acc[j][t];
            __syncthreads();
        }
        if constexpr (LAST) {
            for (int e = tid; e < kThinTile; e += 256) {
                const int i = p.wide ? e % kThin : e / kThin, j = p.wide ? e / kThin : e % kThin;
                if (row0 + i >= p.l || j >= p.s) continue;
                const int64_t at = z * p.batch_o + (p.wide ? j * p.ldo + row0 + i : (row0 + i) * p.ldo + j);
                put_out(p.out, p.bf16, at, p.alpha * y[i * kThinLine + j], p.beta);
            }
        } else {
            for (int e = 4 * tid; e < kThinTile; e += 1024)
                *reinterpret_cast<f32x4 *>(rows + e) = *reinterpret_cast<const f32x4 *>(y + e / kThin * kThinLine + e % kThin);
#pragma unroll 4
            for (int n = 0; n < kThin; n += 4) {
                const float *at = y + (n + low) * kThinLine + r;
                const float x = at[16 * wave];
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x, at[16 * j], sum[j], 0, 0, 0);
            }
        }
        __syncthreads();
    }
    if constexpr (!LAST) {
        float *out = p.gram_out + (z * gridDim.x + blockIdx.x) * kThinTile;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int t = 0; t < 4; ++t) out[(16 * wave + 4 * low + t) * kThin + 16 * j + r] = sum[j][t];
    }
}

// A from its parts, in an order that does not depend on the batch: 8 threads an entry, each every eighth part
__global__ __launch_bounds__(256) void thin_sum_kernel(const float *__restrict__ in, int parts, float *__restrict__ out)
{
    __shared__ float slots[8][32];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    in += (int64_t)blockIdx.z * parts * kThinTile + e;
    float v = 0.0f;
#pragma unroll 8
    for (int k = slice; k < parts; k += 8) v += in[k * kThinTile];
    slots[slice][lane] = v;
    __syncthreads();
    if (slice != 0) return;
    for (int k = 1; k < 8; ++k) v += slots[k][lane];
    out[(int64_t)blockIdx.z * kThinTile + e] = v;
}

struct ThinSpace {
    double *norms;
    float *y, *gram[2], *sum;
    int64_t lp;
    int blocks, chunks;
    size_t bytes;
};
ThinSpace thin_space(uint8_t *base, int64_t batch, int64_t l)
{
    ThinSpace s{};
    s.lp = round_up(l, kThin);
    s.blocks = (int)((s.lp / kThin + kThinChunks - 1) / kThinChunks);
    s.chunks = (int)((s.lp / kThin + s.blocks - 1) / s.blocks);
    auto take = [&](int64_t bytes) {
        uint8_t *p = base ? base + s.bytes : nullptr;
        s.bytes += (size_t)round_up(bytes, 256);
        return p;
    };
    s.norms = reinterpret_cast<double *>(take(8 * kNormBlocks * batch));
    s.y = reinterpret_cast<float *>(take(4 * kThin * s.lp * batch));
    for (int k = 0; k < 2; ++k) s.gram[k] = reinterpret_cast<float *>(take(4 * kThinTile * s.chunks * batch));
    s.sum = reinterpret_cast<float *>(take(4 * kThinTile * batch));
    return s;
}

hipError_t launch_thin(const OrthoProblem &p, const ThinSpace &s, int norm_parts, hipStream_t stream)
{
    Thin t{};
    t.g = p.g;
    t.f32 = p.f32;
    t.bf16 = p.out_bf16;
    t.wide = p.m <= p.n;
    t.s = t.wide ? p.m : p.n;
    t.l = t.wide ? p.n : p.m;
    t.ldg = p.ldg;
    t.batch_g = p.batch_g;
    t.norms = s.norms;
    t.norm_parts = norm_parts;
    t.eps = p.eps;
    t.y = s.y;
    t.lp = s.lp;
    t.blocks = s.blocks;
    t.gram_out = s.gram[0];
    t.a = p.a;
    t.b = p.b;
    t.c = p.c;
    t.alpha = p.alpha;
    t.beta = p.beta;
    t.out = p.out;
    t.ldo = p.ldo;
    t.batch_o = p.batch_o;
    const dim3 grid((unsigned)s.chunks, 1, (unsigned)p.batch), block(256);
    if (p.steps == 0) return launch(thin_kernel<true, true>, grid, block, 0, stream, t);
    hipError_t e = launch(thin_kernel<true, false>, grid, block, 0, stream, t);
    for (int k = 0; k < p.steps && e == hipSuccess; ++k) {
        t.gram = s.gram[k & 1];
        t.parts = s.chunks;
        if (s.chunks > kThinFew) {
            e = launch(thin_sum_kernel, dim3(kThinTile / 32, 1, (unsigned)p.batch), block, 0, stream, t.gram, s.chunks, s.sum);
            if (e) return e;
            t.gram = s.sum;
            t.parts = 1;
        }
        // not where other workgroups of the launch still read
        t.gram_out = s.gram[(k + 1) & 1];
        e = k + 1 < p.steps ? launch(thin_kernel<false, false>, grid, block, 0, stream, t)
                            : launch(thin_kernel<false, true>, grid, block, 0, stream, t);
    }
    return e;
}

// ------------------------------------------------------------------------------ workspace -----
struct Sizes {
    int64_t mp, np, sp, lp;   // rows, columns, shorter and longer side, padded
    slab::Plan gram, poly, update, last;
    size_t partial_bytes;
};
// Every product covers whole tiles of its operands: with 256 x 256 tiles the sides are padded to 256, with
// smaller ones to 128.
Sizes sizes_of(int64_t batch, int64_t m, int64_t n)
{
    Sizes z;
    const auto plans = [&](int64_t pad) {
        z.mp = round_up(m, pad);
        z.np = round_up(n, pad);
        z.sp = m <= n ? z.mp : z.np;
        z.lp = m <= n ? z.np : z.mp;
        z.gram = plan_product(z.sp, z.sp, z.lp / 64, true, batch);
        z.poly = plan_product(z.sp, z.sp, z.sp / 64, true, batch);
        z.update = plan_product(z.mp, z.np, z.sp / 64, false, batch);
        z.last = plan_product(m, n, z.sp / 64, false, batch);
    };
    plans(256);
    const bool big = z.gram.geo == 0 || z.poly.geo == 0 || z.update.geo == 0 || z.last.geo == 0;
    if (!big) {
        plans(128);
        // smaller sides may tip a plan: 256 x 256 tiles need their padding
        if (z.gram.geo == 0 || z.poly.geo == 0 || z.update.geo == 0 || z.last.geo == 0) plans(256);
    }
    z.partial_bytes = std::max(std::max(z.gram.partial_bytes, z.poly.partial_bytes),
                               std::max(z.update.partial_bytes, z.last.partial_bytes));
    return z;
}

struct Space {
    double *part;
    uint16_t *hi[2], *turned[2], *lo, *gram, *poly;
    void *partials;
    size_t bytes;
};
Space carve(uint8_t *base, int64_t batch, const Sizes &z)
{
    Space s{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        uint8_t *p = base ? base + at : nullptr;
        at += (size_t)round_up((int64_t)bytes, 256);
        return p;
    };
    s.part = reinterpret_cast<double *>(take(8 * kNormBlocks * batch));
    const size_t x = (size_t)(2 * batch * z.mp * z.np), a = (size_t)(2 * batch * z.sp * z.sp);
    for (int k = 0; k < 2; ++k) s.hi[k] = reinterpret_cast<uint16_t *>(take(x));
    for (int k = 0; k < 2; ++k) s.turned[k] = reinterpret_cast<uint16_t *>(take(x));
    s.lo = reinterpret_cast<uint16_t *>(take(x));
    s.gram = reinterpret_cast<uint16_t *>(take(a));
    s.poly = reinterpret_cast<uint16_t *>(take(a));
    s.partials = take(z.partial_bytes);
    s.bytes = at;
    return s;
}

template <class Epi>
hipError_t product(const Plan &plan, const Operands &op, const Epi &epi, const Space &s, hipStream_t stream)
{
    return launch_product<F16>(op, epi, plan, s.partials, stream);
}

}  // namespace

size_t ortho_workspace_bytes(int64_t batch, int64_t m, int64_t n)
{
    if (std::min(m, n) <= kThin) return thin_space(nullptr, batch, std::max(m, n)).bytes;
    return carve(nullptr, batch, sizes_of(batch, m, n)).bytes;
}

hipError_t launch_ortho(const OrthoProblem &p, void *ws, hipStream_t stream)
{
    const int64_t esize = p.f32 ? 4 : 2;
    const int vec = p.n % 8 == 0 && (uintptr_t)p.g % 16 == 0 && p.ldg * esize % 16 == 0 && (p.batch == 1 || p.batch_g * esize % 16 == 0);
    const int64_t want = p.m * p.n / kNormTile + 1, most = p.m < kNormBlocks ? p.m : kNormBlocks;
    const int parts = (int)(want < most ? want : most);
    const dim3 ngrid((unsigned)parts, 1, (unsigned)p.batch);
    double *norms = static_cast<double *>(ws);   // first in either workspace
    hipError_t e = p.f32 ? launch(norm_kernel<true>, ngrid, dim3(256), 0, stream, p.g, p.m, p.n, p.ldg, p.batch_g, vec, norms)
                         : launch(norm_kernel<false>, ngrid, dim3(256), 0, stream, p.g, p.m, p.n, p.ldg, p.batch_g, vec, norms);
    if (e) return e;
    if (std::min(p.m, p.n) <= kThin)
        return launch_thin(p, thin_space(static_cast<uint8_t *>(ws), p.batch, std::max(p.m, p.n)), parts, stream);
    const Sizes z = sizes_of(p.batch, p.m, p.n);
    const Space s = carve(static_cast<uint8_t *>(ws), p.batch, z);
    const int64_t bx = z.mp * z.np, ba = z.sp * z.sp;
    const dim3 fgrid((unsigned)(z.mp / 128), (unsigned)(z.np / 128), (unsigned)p.batch);
    e = p.f32 ? launch(first_kernel<true>, fgrid, dim3(256), 0, stream, p.g, p.m, p.n, p.ldg, p.batch_g, vec, s.part, parts, p.eps,
                       s.hi[0], s.lo, s.turned[0], z.mp, z.np, bx)
              : launch(first_kernel<false>, fgrid, dim3(256), 0, stream, p.g, p.m, p.n, p.ldg, p.batch_g, vec, s.part, parts, p.eps,
                       s.hi[0], s.lo, s.turned[0], z.mp, z.np, bx);
    if (e) return e;
    if (p.steps == 0) {
        const int64_t blocks = (p.m * p.n + 255) / 256;
        return launch(copy_out_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536), 1, (unsigned)p.batch), dim3(256), 0,
                      stream, s.hi[0], s.lo, z.np, bx, p.m, p.n, p.alpha, p.beta, p.out, p.out_bf16 ? 1 : 0, p.ldo, p.batch_o);
    }
    const bool wide = p.m <= p.n;
    for (int k = 0; k < p.steps; ++k) {
        const uint16_t *x = s.hi[k & 1], *t = s.turned[k & 1];
        const int after = p.steps - 1 - k;
        const float shift = after < 2 ? std::min(16.0f, std::max(-16.0f, -(p.b + p.c))) / (float)(1 << after) : 0.0f;
        Operands op{};
        // A: rows of X (wide) or of its transpose
        op.a = op.b = reinterpret_cast<const uint8_t *>(wide ? x : t);
        op.lda = op.ldb = 2 * (wide ? z.np : z.mp);
        op.M = op.N = (int)z.sp;
        op.nk = (int)((wide ? z.np : z.mp) / 64);
        op.batch_a = op.batch_b = 2 * bx;
        if ((e = product(z.gram, op, GramEpi{s.gram, z.sp, ba}, s, stream))) return e;
        op.a = op.b = reinterpret_cast<const uint8_t *>(s.gram);
        op.lda = op.ldb = 2 * z.sp;
        op.nk = (int)(z.sp / 64);
        op.batch_a = op.batch_b = 2 * ba;
        if ((e = product(z.poly, op, PolyEpi{s.gram, s.poly, z.sp, ba, p.b, p.c, shift}, s, stream))) return e;
        // the update in X's orientation: poly X for wide, X poly for tall (poly is symmetric)
        op.a = reinterpret_cast<const uint8_t *>(wide ? s.poly : x);
        op.lda = 2 * (wide ? z.sp : z.np);
        op.batch_a = 2 * (wide ? ba : bx);
        op.b = reinterpret_cast<const uint8_t *>(wide ? t : s.poly);
        op.ldb = 2 * (wide ? z.mp : z.sp);
        op.batch_b = 2 * (wide ? bx : ba);
        op.nk = (int)(z.sp / 64);
        op.M = (int)z.mp;
        op.N = (int)z.np;
        if (k + 1 < p.steps) {
            const UpdateEpi epi{x, s.lo, s.hi[(k + 1) & 1], s.turned[(k + 1) & 1], z.np, z.mp, bx, p.a - shift};
            if ((e = product(z.update, op, epi, s, stream))) return e;
        } else {
            op.M = (int)p.m;
            op.N = (int)p.n;
            const float alpha = p.alpha * kUnscale;
            e = p.out_bf16 ? product(z.last, op, LastEpi<true>{x, s.lo, z.np, bx, p.a - shift,
                                                              StoreEpi<true>{p.out, p.ldo, p.batch_o, alpha, p.beta}}, s, stream)
                           : product(z.last, op, LastEpi<false>{x, s.lo, z.np, bx, p.a - shift,
                                                               StoreEpi<false>{p.out, p.ldo, p.batch_o, alpha, p.beta}}, s, stream);
            if (e) return e;
        }
    }
    return hipSuccess;
}

}  // namespace mx
