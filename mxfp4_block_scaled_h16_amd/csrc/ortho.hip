// Newton-Schulz orthogonalisation of a matrix (or a batch of one shape):
//
//   X = G / (|G|_F + eps);  steps times:  A = X X^T,  X <- a X + (b A + c A A) X;  out = alpha X + beta out
//
// with the Gram matrix taken along the shorter side (X^T X for more rows than columns). The
// products run on the FP16 matrix cores with FP32 accumulation. FP16 holds 2^10 X, 2^10 A and
// 2^10 (b A + c A A): every entry of X stays below 1.3 and of the others below 3 in magnitude
// (singular values of X lie in [0, 1.3] at every step for the usual coefficients), so nothing
// overflows, and entries down to 2^-24 keep all 11 bits. X itself is carried from step to step in two FP16
// numbers, value and remainder (22 bits): the term a X, which carries the small singular values,
// loses nothing, and what the 11-bit operands add stays below the rounding of a bf16 result
// (relative error 0.0004 to 0.0016 against bf16's 0.0017; with X in FP16 alone a matrix of a few
// strong directions was off by 0.011, with bf16 operands by 0.09).
//
// Per step three launches: A (symmetric: the lower triangle of tiles, written twice), b A + c A A
// (symmetric too), and the update, which writes X in both orientations for the next step's
// products, each of which contracts along rows.
#include "slab_gemm.h"
#include "train_internal.h"

namespace mx {
namespace {

using namespace slab;

constexpr float kUnscale = 1.0f / 1024.0f;
constexpr float kLoScale = 2048.0f, kLoUnscale = 1.0f / 2048.0f;   // the remainder, held 2^11 larger

__device__ __forceinline__ uint16_t f16_bits(float x) { return __builtin_bit_cast(uint16_t, (_Float16)x); }
__device__ __forceinline__ float f16_float(uint16_t b) { return (float)__builtin_bit_cast(_Float16, b); }
[[maybe_unused]] __device__ __forceinline__ f32x4 f16_quad(const uint16_t *p)
{
    const u32x2 w = *reinterpret_cast<const u32x2 *>(p);
    // copied out first: a bit cast of a vector's element reads the vector's first one
    const uint32_t first = w.x, second = w.y;
    const f16x2 a = __builtin_bit_cast(f16x2, first), b = __builtin_bit_cast(f16x2, second);
    return f32x4{(float)a[0], (float)a[1], (float)b[0], (float)b[1]};
}

// ------------------------------------------------------------------------- the epilogues ------
// A = X X^T: 2^20 A in acc, 2^10 A stored, in both places
struct GramEpi {
    static constexpr bool kSym = true;
    uint16_t *out;
    int64_t ld, batch_out;
    template <class G>
    __device__ __forceinline__ void run(f32x4 (&acc)[G::FI][G::FJ], const Where &w, const Operands &, uint8_t *lds) const
    {
        uint16_t *o = out + w.batch * batch_out;
        store_tile16<G>(w, lds, [](float a, float b) { return pack_f16(a, b); },
                        [&](int i, int j) { return acc[i][j] * kUnscale; },
                        o, ld, w.m0 == w.n0 ? nullptr : o, ld);
    }
};

// b A + c A A: 2^20 A A in acc, 2^10 A read
struct PolyEpi {
    static constexpr bool kSym = true;
    const uint16_t *gram;
    uint16_t *out;
    int64_t ld, batch_out;
    float b, c;
    template <class G>
    __device__ __forceinline__ void run(f32x4 (&acc)[G::FI][G::FJ], const Where &w, const Operands &, uint8_t *lds) const
    {
        const uint16_t *in = gram + w.batch * batch_out;
        uint16_t *o = out + w.batch * batch_out;
        const int r = w.lane & 15, q = w.lane >> 4;
        const float cs = c * kUnscale;
        store_tile16<G>(w, lds, [](float x, float y) { return pack_f16(x, y); },
                        [&](int i, int j) {
                            const f32x4 g =
                                f16_quad(in + (int64_t)(w.m0 + w.row0 + 16 * i + r) * ld + w.n0 + w.col0 + 16 * j + 4 * q);
                            return b * g + cs * acc[i][j];
                        },
                        o, ld, w.m0 == w.n0 ? nullptr : o, ld);
    }
};

// a X + (b A + c A A) X in X's own orientation: value (both orientations) and remainder
struct UpdateEpi {
    static constexpr bool kSym = false;
    const uint16_t *hi;      // X [mp][np]
    uint16_t *lo;            // read and written
    uint16_t *hi_out, *turned;
    int64_t ld, ld_turned, batch_x;
    float a;
    template <class G>
    __device__ __forceinline__ void run(f32x4 (&acc)[G::FI][G::FJ], const Where &w, const Operands &, uint8_t *lds) const
    {
        const int r = w.lane & 15, q = w.lane >> 4;
        const uint16_t *h = hi + w.batch * batch_x;
        uint16_t *l = lo + w.batch * batch_x;
#pragma unroll
        for (int i = 0; i < G::FI; ++i)
#pragma unroll
            for (int j = 0; j < G::FJ; ++j) {
                const int64_t at = (int64_t)(w.m0 + w.row0 + 16 * i + r) * ld + w.n0 + w.col0 + 16 * j + 4 * q;
                const f32x4 x = f16_quad(h + at) + f16_quad(l + at) * kLoUnscale;
                const f32x4 v = a * x + kUnscale * acc[i][j];
                f32x4 rem;
#pragma unroll
                for (int t = 0; t < 4; ++t) rem[t] = (v[t] - f16_float(f16_bits(v[t]))) * kLoScale;
                acc[i][j] = v;
                *reinterpret_cast<u32x2 *>(l + at) = u32x2{pack_f16(rem[0], rem[1]), pack_f16(rem[2], rem[3])};
            }
        store_tile16<G>(w, lds, [](float x, float y) { return pack_f16(x, y); }, [&](int i, int j) { return acc[i][j]; },
                        hi_out + w.batch * batch_x, ld, turned + w.batch * batch_x, ld_turned);
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
    __device__ __forceinline__ void run(f32x4 (&acc)[G::FI][G::FJ], const Where &w, const Operands &op, uint8_t *lds) const
    {
        const int r = w.lane & 15, q = w.lane >> 4;
        const uint16_t *h = hi + w.batch * batch_x, *l = lo + w.batch * batch_x;
        store.template run_with<G>(w, op, lds, [&](int i, int j) {
            const int64_t at = (int64_t)(w.m0 + w.row0 + 16 * i + r) * ld + w.n0 + w.col0 + 16 * j + 4 * q;
            return a * (f16_quad(h + at) + f16_quad(l + at) * kLoUnscale) + kUnscale * acc[i][j];
        });
    }
};

// ----------------------------------------------------------------- norm and first operands ----
constexpr int kNormBlocks = 512;

template <bool F32>
__device__ __forceinline__ float read_g(const void *g, int64_t at)
{
    if constexpr (F32)
        return static_cast<const float *>(g)[at];
    else
        return bf16_float(static_cast<const uint16_t *>(g)[at]);
}

// sums of squares, one per workgroup, in 64 bits (the squares of FP32 numbers leave FP32's range)
template <bool F32>
__global__ __launch_bounds__(256) void norm_kernel(const void *__restrict__ g, int64_t m, int64_t n, int64_t ldg, int64_t batch_g,
                                                   double *__restrict__ part)
{
    __shared__ double slots[4];
    const int64_t base = blockIdx.z * batch_g;
    double sum = 0.0;
    for (int64_t row = blockIdx.x; row < m; row += gridDim.x)
        for (int64_t col = threadIdx.x; col < n; col += 256) {
            const double v = (double)read_g<F32>(g, base + row * ldg + col);
            sum += v * v;
        }
    for (int k = 32; k >= 1; k >>= 1) sum += __shfl_xor(sum, k);
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) part[blockIdx.z * kNormBlocks + blockIdx.x] = (slots[0] + slots[1]) + (slots[2] + slots[3]);
}

// X = G / (|G| + eps), times 2^10, in value and remainder and (the value) transposed, with zeros around it
template <bool F32>
__global__ __launch_bounds__(256) void first_kernel(const void *__restrict__ g, int64_t m, int64_t n, int64_t ldg, int64_t batch_g,
                                                    const double *__restrict__ part, int parts, float eps,
                                                    uint16_t *__restrict__ hi, uint16_t *__restrict__ lo,
                                                    uint16_t *__restrict__ turned, int64_t mp, int64_t np, int64_t batch_x)
{
    __shared__ uint16_t tile[64][64 + 2];
    __shared__ float inv_shared;
    if (threadIdx.x < 64) {
        double sum = 0.0;
        for (int k = threadIdx.x; k < parts; k += 64) sum += part[blockIdx.z * kNormBlocks + k];
        for (int k = 32; k >= 1; k >>= 1) sum += __shfl_xor(sum, k);
        if (threadIdx.x == 0) inv_shared = (float)(1024.0 / (sqrt(sum) + (double)eps));
    }
    __syncthreads();
    const float inv = inv_shared;
    const int64_t r0 = (int64_t)blockIdx.x * 64, c0 = (int64_t)blockIdx.y * 64;
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int64_t r = r0 + ty + 4 * k, c = c0 + tx;
        const float v = r < m && c < n ? read_g<F32>(g, blockIdx.z * batch_g + r * ldg + c) * inv : 0.0f;
        const uint16_t h = f16_bits(v);
        tile[ty + 4 * k][tx] = h;
        if (r < mp && c < np) {
            hi[blockIdx.z * batch_x + r * np + c] = h;
            lo[blockIdx.z * batch_x + r * np + c] = f16_bits((v - f16_float(h)) * kLoScale);
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int64_t c = c0 + ty + 4 * k, r = r0 + tx;
        if (c < np && r < mp) turned[blockIdx.z * batch_x + c * mp + r] = tile[tx][ty + 4 * k];
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
        float v = alpha * ((f16_float(hi[at]) + f16_float(lo[at]) * kLoUnscale) * kUnscale);
        if (bf16) {
            uint16_t *p = static_cast<uint16_t *>(out) + o;
            if (beta != 0.0f) v += beta * bf16_float(*p);
            *p = (uint16_t)(pack_bf16(v, 0.0f) & 0xFFFFu);
        } else {
            float *p = static_cast<float *>(out) + o;
            if (beta != 0.0f) v += beta * *p;
            *p = v;
        }
    }
}

// ------------------------------------------------------------------------------ workspace -----
struct Sizes {
    int64_t mp, np, sp;   // padded rows, columns, shorter side
    bool big;
};
// Tiles of 256 x 256 once the Gram matrix has more of them than half the CUs, else 128 x 128.
Sizes sizes_of(int64_t batch, int64_t m, int64_t n)
{
    const int64_t s = m < n ? m : n, l = m < n ? n : m;
    Sizes z;
    z.big = batch * ((s + 255) / 256) * ((l + 255) / 256) > kComputeUnits / 2;
    const int64_t t = z.big ? 256 : 128;
    z.mp = round_up(m, t);
    z.np = round_up(n, t);
    z.sp = m <= n ? z.mp : z.np;
    return z;
}

struct Space {
    double *part;
    uint16_t *hi[2], *turned[2], *lo, *gram, *poly;
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
    s.bytes = at;
    return s;
}

template <class Epi>
hipError_t product(bool big, const Operands &op, const Epi &epi, int64_t batch, hipStream_t stream)
{
    return big ? launch_product<F16, Big>(op, epi, (int)batch, stream) : launch_product<F16, Small>(op, epi, (int)batch, stream);
}

}  // namespace

size_t ortho_workspace_bytes(int64_t batch, int64_t m, int64_t n)
{
    return carve(nullptr, batch, sizes_of(batch, m, n)).bytes;
}

hipError_t launch_ortho(const OrthoProblem &p, void *ws, hipStream_t stream)
{
    const Sizes z = sizes_of(p.batch, p.m, p.n);
    const Space s = carve(static_cast<uint8_t *>(ws), p.batch, z);
    const int64_t bx = z.mp * z.np, ba = z.sp * z.sp;
    const int parts = (int)(p.m < kNormBlocks ? p.m : kNormBlocks);
    const dim3 ngrid((unsigned)parts, 1, (unsigned)p.batch);
    const dim3 fgrid((unsigned)(z.mp / 64), (unsigned)(z.np / 64), (unsigned)p.batch);
    hipError_t e = p.f32 ? launch(norm_kernel<true>, ngrid, dim3(256), 0, stream, p.g, p.m, p.n, p.ldg, p.batch_g, s.part)
                         : launch(norm_kernel<false>, ngrid, dim3(256), 0, stream, p.g, p.m, p.n, p.ldg, p.batch_g, s.part);
    if (e) return e;
    e = p.f32 ? launch(first_kernel<true>, fgrid, dim3(256), 0, stream, p.g, p.m, p.n, p.ldg, p.batch_g, s.part, parts, p.eps,
                       s.hi[0], s.lo, s.turned[0], z.mp, z.np, bx)
              : launch(first_kernel<false>, fgrid, dim3(256), 0, stream, p.g, p.m, p.n, p.ldg, p.batch_g, s.part, parts, p.eps,
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
        Operands op{};
        // A: rows of X (wide) or of its transpose
        op.a = op.b = reinterpret_cast<const uint8_t *>(wide ? x : t);
        op.lda = op.ldb = 2 * (wide ? z.np : z.mp);
        op.M = op.N = (int)z.sp;
        op.nk = (int)((wide ? z.np : z.mp) / 64);
        op.batch_a = op.batch_b = 2 * bx;
        if ((e = product(z.big, op, GramEpi{s.gram, z.sp, ba}, p.batch, stream))) return e;
        op.a = op.b = reinterpret_cast<const uint8_t *>(s.gram);
        op.lda = op.ldb = 2 * z.sp;
        op.nk = (int)(z.sp / 64);
        op.batch_a = op.batch_b = 2 * ba;
        if ((e = product(z.big, op, PolyEpi{s.gram, s.poly, z.sp, ba, p.b, p.c}, p.batch, stream))) return e;
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
            const UpdateEpi epi{x, s.lo, s.hi[(k + 1) & 1], s.turned[(k + 1) & 1], z.np, z.mp, bx, p.a};
            if ((e = product(z.big, op, epi, p.batch, stream))) return e;
        } else {
            op.M = (int)p.m;
            op.N = (int)p.n;
            const float alpha = p.alpha * kUnscale;
            e = p.out_bf16 ? product(z.big, op, LastEpi<true>{x, s.lo, z.np, bx, p.a,
                                                              StoreEpi<true>{p.out, p.ldo, p.batch_o, alpha, p.beta}},
                                     p.batch, stream)
                           : product(z.big, op, LastEpi<false>{x, s.lo, z.np, bx, p.a,
                                                               StoreEpi<false>{p.out, p.ldo, p.batch_o, alpha, p.beta}},
                                     p.batch, stream);
            if (e) return e;
        }
    }
    return hipSuccess;
}

}  // namespace mx
