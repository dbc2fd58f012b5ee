// 8-bit operands: E4M3 codes with a power-of-two scale for each block of 128 (1 x 128 along the
// contraction, or 128 x 128), and their product on the scaled FP8 matrix cores.
#include "mx_device.h"
#include "slab_gemm.h"
#include "train_internal.h"

namespace mx {
namespace {

// ------------------------------------------------------------------------------ quantizer -----
// One workgroup quantizes a 128 x 128 tile of x, which holds whole blocks along both axes; 256 threads of
// 8 x 8 values each (rows 8 (t / 16) .., columns 8 (t % 16) ..), in registers throughout. Row
// maxima join the 16 lanes of a row, column maxima the 16 threads of a column through the LDS.
// Bound by memory: a bf16 value is read once (2 bytes) and a code written per axis (1 byte each). 8192 x 4096 and
// 6144 x 4096 along their rows in one launch: 39 us, 4.5 TB/s of the 4.97 that a copy reaches; 8192 x 14336 and 8192 x
// 4096 along their columns: 102 us, 4.4 TB/s.
struct Fp8Args {
    Fp8Input item[kFp8Group];
    int first[kFp8Group + 1];   // workgroups before each item
    int tiles_n[kFp8Group];
};

// E8M0 byte of a block from the bit pattern of its largest magnitude: the smallest S with
// amax <= 448 * 2^(S - 127); 448 = 1.75 * 2^8, so the exponent less 8, one more above 1.75.
// 0xFF: the block holds a NaN or infinity.
__device__ __forceinline__ uint32_t e8m0_of(uint32_t amax)
{
    if (amax >= 0x7F800000u) return 0xFFu;
    const int s = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(s, 0);
}

// Four values times 2^(127 - S) (exact: a power of two, S <= 247) as E4M3 codes, rounded to nearest
// even by the conversion; the product is at most 448.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv)
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
    return (uint32_t)w;
}
// 2^(127 - S), S in [0, 247]: exponent field 254 - S
__device__ __forceinline__ float inverse_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
// the maximum over the 16 lanes of a row, in each of them
__device__ __forceinline__ uint32_t row16_max(uint32_t v)
{
    v = max(v, dpp<0xB1>(v));    // quad_perm [1,0,3,2]
    v = max(v, dpp<0x4E>(v));    // quad_perm [2,3,0,1]
    v = max(v, dpp<0x141>(v));   // row_half_mirror
    return max(v, dpp<0x140>(v));  // row_mirror
}

// rows that are aligned to their elements only: the 16-byte loads then go to any even address, which
// gfx950 serves (unaligned access is on for every HIP process), at up to twice the lines a load
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <bool F32>
__device__ __forceinline__ float load1(const Fp8Input &it, int64_t at)
{
    if constexpr (F32)
        return static_cast<const float *>(it.x)[at];
    else
        return bf16_lo(static_cast<const uint16_t *>(it.x)[at]);
}

// RAGGED: a row may end within these eight
template <bool F32, bool RAGGED>
__device__ __forceinline__ void load8(const Fp8Input &it, int64_t row, int64_t col, float (&v)[8])
{
    if (row < it.rows && (RAGGED ? col + 8 <= it.cols : col < it.cols)) {
        if constexpr (F32) {
            const float *p = static_cast<const float *>(it.x) + row * it.ldx + col;
            const f32x4 a = *reinterpret_cast<const f32x4_any *>(p), b = *reinterpret_cast<const f32x4_any *>(p + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = a[e];
                v[4 + e] = b[e];
            }
        } else {
            const u32x4 a =
                *reinterpret_cast<const u32x4_any *>(static_cast<const uint16_t *>(it.x) + row * it.ldx + col);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = bf16_lo(a[e]);
                v[2 * e + 1] = bf16_hi(a[e]);
            }
        }
        return;
    }
    // the end of a row, value by value
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = 0.0f;
        if constexpr (RAGGED)
            if (row < it.rows && col + e < it.cols) v[e] = load1<F32>(it, row * it.ldx + col + e);
    }
}

// F32: the tensors' type. RAGGED: some row's length is no multiple of eight (its end is then read value by
// value, in code that the others need not fetch). Four workgroups a CU (128 registers) instead of three, where that
// spills nothing: 8192 x (14336 + 4096) along the columns 118 -> 101 us; with five, or in the ragged ones, it spills
// (1111 x 2001 and 2001 x 1000: 12 -> 18 us).
template <bool F32, bool RAGGED>
__global__ __launch_bounds__(256, RAGGED ? 2 : 4) void fp8_quantize_kernel(Fp8Args args)
{
    __shared__ uint32_t cmax[16][128 + 4];
    __shared__ uint32_t wmax[4];
    // a column's 128 codes: 16 pieces of 8 bytes, permuted by the column's bits 3-6 against bank conflicts
    __shared__ __attribute__((aligned(16))) uint8_t tr[128 * 128];
    const int which = (int)blockIdx.x >= args.first[1] ? 1 : 0;
    const Fp8Input &it = args.item[which];
    const int block = (int)blockIdx.x - args.first[which];
    const int64_t tm = block / args.tiles_n[which], tn = block % args.tiles_n[which];
    const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
    const int64_t row0 = tm * 128 + 8 * rg, col0 = tn * 128 + 8 * cg;

    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) load8<F32, RAGGED>(it, row0 + i, col0, v[i]);
    uint32_t rmax[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rmax[i] = row16_max(amax_bits<8>(v[i]));
    uint32_t tile_s = 0;
    if (it.tile) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, rmax[i]);
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if ((tid & 63) == 0) wmax[tid >> 6] = m;
        __syncthreads();
        tile_s = e8m0_of(max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3])));
    }
    if (it.axis1.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t row = row0 + i;
            if (row >= it.rows) break;
            const uint32_t s = it.tile ? tile_s : e8m0_of(rmax[i]);
            const float inv = inverse_scale(s == 0xFFu ? 0u : s);
            slab::u32x2 w = {0u, 0u};
            if (s != 0xFFu)
                w = slab::u32x2{encode4(v[i][0], v[i][1], v[i][2], v[i][3], inv),
                                encode4(v[i][4], v[i][5], v[i][6], v[i][7], inv)};
            *reinterpret_cast<slab::u32x2 *>(it.axis1.q + row * it.axis1.ldq + col0) = w;
            if (cg == 0) it.axis1.s[row * it.axis1.lds + tn] = (uint8_t)s;
        }
    }
    if (it.axis0.q) {
        if (!it.tile) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i][j]));
                cmax[rg][8 * cg + j] = m;
            }
            __syncthreads();
            if (tid < 128) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) m = max(m, cmax[i][tid]);
                cmax[0][tid] = e8m0_of(m);
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int col = 8 * cg + j;
            const uint32_t s = it.tile ? tile_s : cmax[0][col];
            const float inv = inverse_scale(s == 0xFFu ? 0u : s);
            slab::u32x2 w = {0u, 0u};
            if (s != 0xFFu)
                w = slab::u32x2{encode4(v[0][j], v[1][j], v[2][j], v[3][j], inv),
                                encode4(v[4][j], v[5][j], v[6][j], v[7][j], inv)};
            *reinterpret_cast<slab::u32x2 *>(tr + col * 128 + 8 * (rg ^ (col >> 3))) = w;
        }
        __syncthreads();
        // 8 lanes write a column's 128 bytes
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int col = 32 * p + (tid >> 3), piece = 2 * (tid & 7);
            const int64_t out = tn * 128 + col;
            if (out >= it.cols) continue;
            const slab::u32x2 lo = *reinterpret_cast<const slab::u32x2 *>(tr + col * 128 + 8 * (piece ^ (col >> 3)));
            const slab::u32x2 hi =
                *reinterpret_cast<const slab::u32x2 *>(tr + col * 128 + 8 * ((piece + 1) ^ (col >> 3)));
            *reinterpret_cast<u32x4 *>(it.axis0.q + out * it.axis0.ldq + tm * 128 + 8 * piece) =
                u32x4{lo.x, lo.y, hi.x, hi.y};
            if ((tid & 7) == 0)
                it.axis0.s[out * it.axis0.lds + tm] = (uint8_t)(it.tile ? tile_s : cmax[0][col]);
        }
    }
}

__global__ __launch_bounds__(256) void scale_output_kernel(void *c, int bf16, int64_t M, int64_t N, int64_t ldc, float beta)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < M * N; i += (int64_t)gridDim.x * 256) {
        const int64_t at = i / N * ldc + i % N;
        if (bf16) {
            uint16_t *p = static_cast<uint16_t *>(c) + at;
            *p = beta == 0.0f ? (uint16_t)0 : (uint16_t)(slab::pack_bf16(beta * slab::bf16_float(*p), 0.0f) & 0xFFFFu);
        } else {
            float *p = static_cast<float *>(c) + at;
            *p = beta == 0.0f ? 0.0f : beta * *p;
        }
    }
}

}  // namespace

hipError_t launch_scale_output(void *c, bool bf16, int64_t M, int64_t N, int64_t ldc, float beta, hipStream_t stream)
{
    const int64_t blocks = (M * N + 255) / 256;
    return launch(scale_output_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, stream, c,
                  bf16 ? 1 : 0, M, N, ldc, beta);
}

hipError_t launch_fp8_quantize(const Fp8Input *items, int count, hipStream_t stream)
{
    Fp8Args args{};
    int64_t total = 0;
    int n = 0;
    for (int i = 0; i < count; ++i) {
        if (items[i].rows == 0 || items[i].cols == 0) continue;
        args.item[n] = items[i];
        args.first[n] = (int)total;
        args.tiles_n[n] = (int)((items[i].cols + 127) / 128);
        total += (items[i].rows + 127) / 128 * args.tiles_n[n];
        ++n;
    }
    if (n == 0) return hipSuccess;
    if (total > kFp8Tiles) return hipErrorInvalidValue;
    for (int i = n; i <= kFp8Group; ++i) args.first[i] = (int)total;
    bool ragged = false;
    for (int i = 0; i < n; ++i) ragged = ragged || args.item[i].cols % 8 != 0;
    const dim3 grid((unsigned)total), block(256);
    if (args.item[0].f32)
        return ragged ? launch(fp8_quantize_kernel<true, true>, grid, block, 0, stream, args)
                      : launch(fp8_quantize_kernel<true, false>, grid, block, 0, stream, args);
    return ragged ? launch(fp8_quantize_kernel<false, true>, grid, block, 0, stream, args)
                  : launch(fp8_quantize_kernel<false, false>, grid, block, 0, stream, args);
}

size_t fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    return slab::plan_product(M, N, round_up(K, 128) / 128, false, 1).partial_bytes;
}

hipError_t launch_fp8_gemm(const uint8_t *aq, int64_t lda, const uint8_t *as, int64_t ldas, const uint8_t *bq,
                           int64_t ldb, const uint8_t *bs, int64_t ldbs, int64_t M, int64_t N, int64_t K, float alpha,
                           float beta, void *c, bool bf16, int64_t ldc, void *workspace, size_t ws_bytes,
                           hipStream_t stream)
{
    using namespace slab;
    Operands op{};
    op.a = aq;
    op.b = bq;
    op.lda = lda;
    op.ldb = ldb;
    op.as = as;
    op.bs = bs;
    op.ldas = ldas;
    op.ldbs = ldbs;
    op.M = (int)M;
    op.N = (int)N;
    op.nk = (int)(round_up(K, 128) / 128);
    Plan plan = plan_product(M, N, op.nk, false, 1);
    if (plan.partial_bytes > ws_bytes || !workspace) plan = unsplit(plan, op.nk);
    auto run = [&](const auto &epi) { return launch_product<E4M3>(op, epi, plan, workspace, stream); };
    return bf16 ? run(StoreEpi<true>{c, ldc, 0, alpha, beta}) : run(StoreEpi<false>{c, ldc, 0, alpha, beta});
}

}  // namespace mx
