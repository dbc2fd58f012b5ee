// Softmax cross entropy of a linear head, in pieces of the vocabulary, without keeping the logits.
//
//   z = X W^T,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,target
//   G_tv = exp(z_tv - lse_t) (dloss_t + dlse_t) - [v = target_t] dloss_t,  dX = G W,  dW = G^T X
//
// Forward: one product whose epilogue leaves a maximum and a sum of exponentials per row and
// column tile, and a kernel that joins them. Backward: for each piece of the vocabulary the logits
// are formed again and leave the product's epilogue as G, in FP16 (scaled to its range) and in both
// orientations; dX = G W adds up over the pieces in FP32, dW = G^T X has its rows of the piece written
// once. The second operands of these are FP16 copies of W's piece and of X, transposed, so that every
// product contracts along rows.
//
// Bound by the matrix cores, under the card's power cap: at T 8192, K 4096, V 128256 26.9 ms, of which the loss' product
// 6.14 (1.40 PFLOP/s; the library's plain product, which stores its logits, 5.8 in turn with it), and in each of eight
// pieces G's 0.89, dX's 0.85 and dW's 0.78 (1.21, 1.26 and 1.38 PFLOP/s). At T 2048, K 2048, V 50257 the loss takes 376 us, of
// which the product 354 and the joining of its rows and of its last tiles 10 each; the library's product alone, in turn
// with it, 401 to 370. What is not products: 3% at the large size (copies 49 us a piece, ranges 0.2 ms), at T 1537, K 1024 a
// tenth of 0.87 ms; at T 128, K 512, V 1000 a call's 42 us are 7 launches one after the other, of 3 to 6 us. (Kernels and
// wholes from one session, 20 to 60 calls on end.)
#include <algorithm>
#include <cfloat>

#include "mx_device.h"
#include "slab_gemm.h"
#include "train_internal.h"

namespace mx {
namespace {

using namespace slab;

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// ------------------------------------------------------------------------ the loss' product ---
// Per row of the tile: the largest z and the sum of exp(z - largest) over the tile's columns
// and the target's z where the tile holds it. A lane holds 16
// columns of a row per 16-row tile, the lanes 16, 32 and 48 further the others of the wavefront's 64;
// the wavefronts of a row join through the LDS.
struct StatsEpi {
    static constexpr bool kSym = false;
    float2 *part;            // [tiles_n][T]
    float *zt;               // [T]
    const int64_t *target;
    int64_t v0;              // the launch's first column

    template <class G>
    __device__ __forceinline__ void run(f32x4 (&acc)[G::FI][G::FJ], const Where &w, const Operands &op, uint8_t *lds,
                                        uint8_t *) const
    {
        const int r = w.lane & 15, q = w.lane >> 4;
        float2 *slots = reinterpret_cast<float2 *>(lds);   // [wave column][row of the tile]
        const int wn = w.wave / G::kWavesM;
        const int nleft = op.N - (w.n0 + w.col0 + 4 * q);   // valid: 16 j + t < nleft
#pragma unroll
        for (int i = 0; i < G::FI; ++i) {
            if (i / 2 < w.block0 || i / 2 >= w.block1) continue;
            const int row = w.row0 + 16 * i + r;
            const int m = min(w.m0 + row, op.M - 1);
            // the target's place among this lane's columns; far outside when it is not an index
            const int64_t tc = target[m] - v0 - (w.n0 + w.col0 + 4 * q);
            const int want = tc >= 0 && tc < 64 ? (int)tc : -1;
            float top = -INFINITY;
            float hit = 0.0f;
            bool found = false;
#pragma unroll
            for (int j = 0; j < G::FJ; ++j)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int c = 16 * j + t;
                    float z = acc[i][j][t];
                    if (c == want) {
                        hit = z;
                        found = true;
                    }
                    z = c < nleft ? z : -INFINITY;
                    acc[i][j][t] = z;
                    top = fmaxf(top, z);
                }
            if (found && w.m0 + row < op.M && want < nleft) zt[m] = hit;
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float ref = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < G::FJ; ++j)
#pragma unroll
                for (int t = 0; t < 4; ++t) sum += fast_exp2((acc[i][j][t] - ref) * kLog2e);
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (q == 0) slots[wn * G::kTileM + row] = make_float2(top, sum);
        }
        __syncthreads();
        for (int row = threadIdx.x; row < G::kTileM; row += 64 * G::NW) {
            const int blk = row % G::kWaveRows / G::kBlockRows;
            if (blk < w.block0 || blk >= w.block1) continue;
            float2 s = slots[row];
#pragma unroll
            for (int k = 1; k < G::kWavesN; ++k) {
                const float2 o = slots[k * G::kTileM + row];
                const float top = fmaxf(s.x, o.x), ref = top == -INFINITY ? 0.0f : top;
                s = make_float2(top, s.y * fast_exp2((s.x - ref) * kLog2e) + o.y * fast_exp2((o.x - ref) * kLog2e));
            }
            const int m = w.m0 + row;
            if (m < op.M) part[(int64_t)(w.n0 / G::kTileN) * op.M + m] = s;
        }
    }
};

// Joins the column tiles of 32 rows: 8 threads per row, each every eighth tile. Few bytes (8 a row and tile), read
// with a wait after each step: 10 us at 2048 rows of 197 tiles, 31 at 8192 of 501.
__global__ __launch_bounds__(256) void xent_join_kernel(const float2 *__restrict__ part, int tiles, int T, int64_t V,
                                                        const float *__restrict__ zt, const int64_t *__restrict__ target,
                                                        int64_t ignore_index, float *__restrict__ loss,
                                                        float *__restrict__ lse)
{
    __shared__ float2 slots[8][32];
    const int lr = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int t = blockIdx.x * 32 + lr;
    auto join = [](float2 s, float2 o) {
        const float top = fmaxf(s.x, o.x), ref = top == -INFINITY ? 0.0f : top;
        return make_float2(top, s.y * fast_exp2((s.x - ref) * kLog2e) + o.y * fast_exp2((o.x - ref) * kLog2e));
    };
    float2 s = make_float2(-INFINITY, 0.0f);
    if (t < T)
        for (int k = slice; k < tiles; k += 8) s = join(s, part[(int64_t)k * T + t]);
    slots[slice][lr] = s;
    __syncthreads();
    if (slice != 0 || t >= T) return;
    for (int k = 1; k < 8; ++k) s = join(s, slots[k][lr]);
    // the loss not from lse: a confident row's is small beside it
    const float rest = log2f(s.y) * kLn2;
    lse[t] = s.x + rest;
    const int64_t tg = target[t];
    float v = 0.0f;
    if (tg != ignore_index) v = tg >= 0 && tg < V ? s.x - zt[t] + rest : NAN;
    loss[t] = v;
}

// -------------------------------------------------------------------- the gradient's product --
// How far the FP16 operands of the gradients' products are scaled: the exponents of powers of two that bring the
// largest finite |G|, |X| and |W| to [2^14, 2^15), and what undoes them in dX and dW. A NaN or an infinity does not
// count: it stays what it is at any scale, and so takes no bits from the other rows or words.
struct Ranges {
    int g, x, w;
    int up_gw, up_gx;   // -(g + w) and -(g + x)
};

// k with 2^14 <= 2^k top < 2^15; 0 for zero. top is finite.
__device__ __forceinline__ int range_shift(float top) { return top > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(top) : 0; }

// Which rows of X add something to the gradients: the others are taken as zeros in the transposed
// copy, so that what a padded position holds (a NaN) meets no zero of G.
struct RowWeights {
    const float *dloss, *dlse;   // NULL: zeros
    const int64_t *target;       // NULL: every row counts
    int64_t ignore_index, V;
    // the gradients of the row's loss and of the row's exponentials
    __device__ __forceinline__ void of(int64_t t, float &dl, float &dp) const
    {
        const int64_t tg = target[t];
        dl = dloss && tg != ignore_index && tg >= 0 && tg < V ? dloss[t] : 0.0f;
        dp = dl + (dlse ? dlse[t] : 0.0f);
    }
    __device__ __forceinline__ bool live(int64_t t) const
    {
        if (!target) return true;
        float dl, dp;
        of(t, dl, dp);
        return dl != 0.0f || dp != 0.0f;
    }
};

// G of the tile, scaled to FP16's range and rounded to it once (11 bits: an eighth of what a bf16 result
// loses in its own rounding), zero in rows past T and in columns past V.
struct GradEpi {
    static constexpr bool kSym = false;
    RowWeights weights;
    const float *lse;
    int64_t v0;                    // the piece's first column
    const Ranges *ranges;
    uint16_t *g, *gt;              // [Tp][ldg], [Vc][ldt]
    int64_t ldg, ldt;

    template <class G>
    __device__ __forceinline__ void run(f32x4 (&acc)[G::FI][G::FJ], const Where &w, const Operands &op, uint8_t *lds,
                                        uint8_t *info_at) const
    {
        // of each row of the tile: scaled dl and dp, lse, and the target's column in the piece (-1: no
        // column of it, or a row without a gradient of its loss)
        f32x4 *info = reinterpret_cast<f32x4 *>(info_at);
        const int up = ranges->g;
        for (int row = threadIdx.x; row < G::kTileM; row += 64 * G::NW) {
            const int m = w.m0 + row;
            f32x4 v = {0.0f, 0.0f, 0.0f, __int_as_float(-1)};
            if (m < op.M) {
                float dl, dp;
                weights.of(m, dl, dp);
                const int64_t at = weights.target[m] - v0;
                v = f32x4{ldexpf(dl, up), ldexpf(dp, up), lse[m],
                          __int_as_float(dl != 0.0f && at >= 0 && at < op.N ? (int)at : -1)};
            }
            info[row] = v;
        }
        __syncthreads();
        store_tile16<G>(acc, w, lds, [](float a, float b) { return pack_f16(a, b); },
                        [&](int m, int) { return info[m - w.m0]; },
                        [&](f32x4 (&z)[2], const f32x4 &row, int, int n) {
                            const float dl = row[0], dp = row[1], ref = row[2];
                            const int want = __float_as_int(row[3]) - n, left = op.N - n;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                // z - lse first: it is exact where the two are close, so that p is 1 as nearly as
                                // lse tells, and p - 1 at a confident row's target no remainder of lse log2(e)
                                float v = fast_exp2((z[e / 4][e % 4] - ref) * kLog2e) * dp;
                                // dp == 0: nothing of the exponentials counts, whatever they are
                                v = e < left && dp != 0.0f ? v : 0.0f;
                                z[e / 4][e % 4] = e == want ? v - dl : v;
                            }
                        },
                        g, ldg, gt, ldt);
    }
};

// ---------------------------------------------------------------------------- ranges ----------
constexpr int kRangeBlocks = 1024;   // at most so many partial maxima, of each of the three
constexpr int kRangeChunk = 8192;    // values of a row that a workgroup takes at a time

__device__ __forceinline__ float block_max(float v)
{
    __shared__ float slots[4];
    for (int k = 32; k >= 1; k >>= 1) v = fmaxf(v, __shfl_xor(v, k));
    __syncthreads();   // slots may still be read from the call before
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    return fmaxf(fmaxf(slots[0], slots[1]), fmaxf(slots[2], slots[3]));
}

// Largest finite |value| of a bf16 matrix over this workgroup's share of it. The magnitudes' bits are moved up
// by 0x80, which carries those of NaN and infinity (0x7F80 and above) into the sign: as signed numbers they are
// below every finite one, two values an instruction.
// Bound by memory, 2 bytes a value: 8192 x 4096 and 128256 x 4096 in 208 us, 5.4 TB/s. vec: 16-byte aligned rows of whole
// 16 bytes.
__device__ __forceinline__ float share_max(const uint16_t *p, int64_t ld, int64_t rows, int64_t cols, bool vec,
                                           const RowWeights &weights)
{
    const int tid = threadIdx.x;
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    s16x2 most = {0x80, 0x80};
    const auto see = [&](uint32_t w) {
        const u16x2 up = __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu) + (unsigned short)0x80;
        most = __builtin_elementwise_max(most, __builtin_bit_cast(s16x2, up));
    };
    if (vec && !weights.target && ld == cols) {   // one row of everything
        const int64_t n = rows * cols / 8, step = (int64_t)gridDim.x * 256;
        int64_t i = (int64_t)blockIdx.x * 256 + tid;
        for (; i + 3 * step < n; i += 4 * step) {
            u32x4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = *reinterpret_cast<const u32x4 *>(p + (i + u * step) * 8);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) see(v[u][e]);
        }
        for (; i < n; i += step) {
            const u32x4 v = *reinterpret_cast<const u32x4 *>(p + i * 8);
#pragma unroll
            for (int e = 0; e < 4; ++e) see(v[e]);
        }
    } else {
        const int64_t chunks = (cols + kRangeChunk - 1) / kRangeChunk;
        for (int64_t b = blockIdx.x; b < rows * chunks; b += gridDim.x) {
            const int64_t row = chunks == 1 ? b : b / chunks, c0 = chunks == 1 ? 0 : (b - row * chunks) * kRangeChunk;
            if (!weights.live(row)) continue;
            const int64_t end = c0 + kRangeChunk < cols ? c0 + kRangeChunk : cols;
            const uint16_t *src = p + row * ld;
            if (vec)
                for (int64_t c = c0 + 8 * tid; c < end; c += 2048) {
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(src + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) see(v[e]);
                }
            else
                for (int64_t c = c0 + tid; c < end; c += 256) see(src[c]);
        }
    }
    return __uint_as_float((uint32_t)(max((int)most[0], (int)most[1]) - 0x80) << 16);
}

// part[0 ..]: the largest |dloss| + |dloss + dlse| of finite ones, part[kRangeBlocks ..]: |X| in live rows, then |W|
__global__ __launch_bounds__(256) void range_kernel(const uint16_t *x, int64_t ldx, const uint16_t *w, int64_t ldw, int64_t T,
                                                    int64_t K, int64_t V, int vec, RowWeights weights, float *part)
{
    float top = 0.0f;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < T; t += (int64_t)gridDim.x * 256) {
        float dl, dp;
        weights.of(t, dl, dp);
        // two finite numbers may add up to infinity
        if (fabsf(dl) < INFINITY && fabsf(dp) < INFINITY) top = fmaxf(top, fminf(fabsf(dl) + fabsf(dp), FLT_MAX));
    }
    const float g = block_max(top);
    const float tx = block_max(share_max(x, ldx, T, K, vec, weights));
    const float tw = block_max(share_max(w, ldw, V, K, vec, RowWeights{}));
    if (threadIdx.x == 0) {
        part[blockIdx.x] = g;
        part[kRangeBlocks + blockIdx.x] = tx;
        part[2 * kRangeBlocks + blockIdx.x] = tw;
    }
}

// The scales, from the partial maxima: by every workgroup of the first kernel that needs them, the first of which
// leaves them for those that follow.
__device__ __forceinline__ Ranges join_ranges(const float *part, int blocks)
{
    __shared__ float slots[3][4];
    float s[3] = {0.0f, 0.0f, 0.0f};
    for (int i = threadIdx.x; i < blocks; i += 256)
#pragma unroll
        for (int k = 0; k < 3; ++k) s[k] = fmaxf(s[k], part[k * kRangeBlocks + i]);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        for (int d = 32; d >= 1; d >>= 1) s[k] = fmaxf(s[k], __shfl_xor(s[k], d));
        if ((threadIdx.x & 63) == 0) slots[k][threadIdx.x >> 6] = s[k];
    }
    __syncthreads();
    int e[3];
#pragma unroll
    for (int k = 0; k < 3; ++k)
        e[k] = range_shift(fmaxf(fmaxf(slots[k][0], slots[k][1]), fmaxf(slots[k][2], slots[k][3])));
    return Ranges{e[0], e[1], e[2], -(e[0] + e[2]), -(e[0] + e[1])};
}

// ------------------------------------------------------------------------------- copies -------
// A matrix to be transposed and scaled: out[c][r] = in[r][c] * scale, bf16 to FP16; r < rows (zero for rows up to
// rows_padded, a multiple of 64, and for rows that add nothing), c < cols. in == NULL: none.
struct Turn {
    const uint16_t *in;
    int64_t ld_in, rows, cols;
    uint16_t *out;
    int64_t ld_out, rows_padded;
    int vec, across;   // 16-byte aligned rows; tiles across the columns
    int tiles;
};
// One or two of them, X's and that of a piece of W. 128 x 128 tiles: a thread transposes 8 x 8 values in
// registers, then 256-byte lines are put together in the LDS. Bound by memory: 2 bytes in, 2 out; a piece of 16128 x
// 4096 in 49 us, 5.4 TB/s.
// blocks > 0: the ranges are joined here.
__global__ __launch_bounds__(256) void turn_kernel(Turn tx, Turn tw, RowWeights weights, const float *part, int blocks,
                                                   Ranges *ranges)
{
    __shared__ __attribute__((aligned(16))) uint16_t tile[128 * 128];   // [column][row], 16-byte pieces permuted
    const bool is_w = (int)blockIdx.x >= tx.tiles;
    const Turn &t = is_w ? tw : tx;
    const int index = (int)blockIdx.x - (is_w ? tx.tiles : 0);
    const int64_t rows = t.rows, cols = t.cols, ld_in = t.ld_in, ld_out = t.ld_out, rows_padded = t.rows_padded;
    const uint16_t *in = t.in;
    uint16_t *out = t.out;
    const int vec = t.vec;
    if (is_w) weights.target = nullptr;   // every row of W counts
    const int64_t r0 = (int64_t)(index / t.across) * 128, c0 = (int64_t)(index % t.across) * 128;
    const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    u32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 8 * rg + i, c = c0 + 8 * cg;
        v[i] = u32x4{0u, 0u, 0u, 0u};
        if (r < rows && weights.live(r)) {
            const uint16_t *p = in + r * ld_in + c;
            if (vec && c + 8 <= cols) {
                v[i] = *reinterpret_cast<const u32x4 *>(p);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < cols) v[i][e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
            }
        }
    }
    // behind the loads, whose wait it shares
    Ranges now;
    if (blocks > 0) {
        now = join_ranges(part, blocks);
        if (blockIdx.x == 0 && threadIdx.x == 0) *ranges = now;
    } else {
        now = *ranges;
    }
    const int up = is_w ? now.w : now.x;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        u32x4 o;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t a = v[2 * k][e / 2], b = v[2 * k + 1][e / 2];
            o[k] = e & 1 ? pack_f16(ldexpf(bf16_hi(a), up), ldexpf(bf16_hi(b), up))
                         : pack_f16(ldexpf(bf16_lo(a), up), ldexpf(bf16_lo(b), up));
        }
        const int c = 8 * cg + e;
        *reinterpret_cast<u32x4 *>(tile + c * 128 + 8 * (rg ^ (cg & 15))) = o;
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int c = 16 * p + (threadIdx.x >> 4), piece = threadIdx.x & 15;
        const int64_t oc = c0 + c, r = r0 + 8 * piece;
        if (oc < cols && r < rows_padded)
            *reinterpret_cast<u32x4 *>(out + oc * ld_out + r) =
                *reinterpret_cast<const u32x4 *>(tile + c * 128 + 8 * (piece ^ ((c >> 3) & 15)));
    }
}

// out[r][c] = in[r][c] (16-bit), zero for cols <= c < ld_out
__global__ __launch_bounds__(256) void pad16_kernel(const uint16_t *__restrict__ in, int64_t ld_in, int64_t rows, int64_t cols,
                                                    uint16_t *__restrict__ out, int64_t ld_out)
{
    const int64_t total = rows * ld_out;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / ld_out, c = i % ld_out;
        out[i] = c < cols ? in[r * ld_in + c] : (uint16_t)0;
    }
}

Turn turn_of(const void *in, int64_t ld_in, int64_t rows, int64_t cols, uint16_t *out, int64_t ld_out, int64_t rows_padded)
{
    Turn t{};
    t.in = static_cast<const uint16_t *>(in);
    t.ld_in = ld_in;
    t.rows = rows;
    t.cols = cols;
    t.out = out;
    t.ld_out = ld_out;
    t.rows_padded = rows_padded;
    t.vec = (uintptr_t)in % 16 == 0 && ld_in % 8 == 0;
    t.across = (int)((cols + 127) / 128);
    t.tiles = (int)((rows_padded + 127) / 128) * t.across;
    return t;
}

// ------------------------------------------------------------------------------ workspace -----
// Pieces of the vocabulary, as even as whole tiles allow: of as many columns as give G 256 MB per orientation, which
// stays near the last-level cache, but of 2048 before they are evened out if that is more (1280 columns at T 70000, V 2100;
// from 65536 tokens on G is larger: 8 GB at 2^21).
int64_t piece_columns(int64_t T, int64_t V)
{
    const int64_t tp = round_up(T, 256);
    int64_t most = ((int64_t)1 << 27) / tp / 256 * 256;
    if (most < 2048) most = 2048;
    const int64_t pieces = (V + most - 1) / most;
    return round_up((V + pieces - 1) / pieces, 256);
}

// The loss keeps no logits, so its tiles may be more than a grid holds: then a launch takes as many columns
// of the vocabulary as make 2^23 - 1 tiles of 256 x 256. part holds the launches' tiles one after the other.
int64_t loss_columns(int64_t T, int64_t V)
{
    const int64_t most = kMaxItems / kThreads[0] / ((T + 255) / 256) * 256;
    return V < most ? V : most;
}
Plan loss_plan(int64_t T, int64_t K, int64_t cols) { return plan_product(T, cols, round_up(K, 64) / 64, false, 1); }
int64_t loss_tiles(const Plan &plan, int64_t cols) { return (cols + kTileSide[plan.geo] - 1) / kTileSide[plan.geo]; }

// The products of a piece: G covers whole tiles, and the products over it run to the end of the last one.
struct PiecePlans {
    Plan g, dx, dw;
    int64_t cols_done, rows_done;
};
PiecePlans plans_of(int64_t T, int64_t K, int64_t cols)
{
    PiecePlans p;
    p.g = plan_product(T, cols, round_up(K, 64) / 64, false, 1);
    const int64_t side = kTileSide[p.g.geo];
    p.cols_done = round_up(cols, side);
    p.rows_done = round_up(T, side);
    p.dx = plan_product(T, K, p.cols_done / 64, false, 1);
    p.dw = plan_product(cols, K, p.rows_done / 64, false, 1);
    return p;
}

struct Carve {
    uint8_t *base;
    size_t at = 0;
    void *take(size_t bytes)
    {
        void *p = base ? base + at : nullptr;
        at += (size_t)round_up((int64_t)bytes, 256);
        return p;
    }
};

struct Layout {
    uint16_t *xp, *wp;   // copies of X and W with rows padded to whole stages (K % 64 != 0)
    float2 *part;
    float *zt;
    float *range_part;
    Ranges *ranges;
    uint16_t *xt, *wt, *g, *gt;
    float *dx;
    void *partials;      // of products whose contraction is split
};
Layout carve(Carve &c, int64_t T, int64_t K, int64_t V, bool backward)
{
    Layout l{};
    const int64_t kp = round_up(K, 64);
    if (K % 64 != 0) {
        l.xp = static_cast<uint16_t *>(c.take(2 * T * kp));
        l.wp = static_cast<uint16_t *>(c.take(2 * V * kp));
    }
    if (!backward) {
        const int64_t step = loss_columns(T, V), rest = V % step;
        const Plan plan = loss_plan(T, K, step);
        int64_t tiles = V / step * loss_tiles(plan, step);
        size_t most = plan.partial_bytes;
        if (rest) {
            const Plan end = loss_plan(T, K, rest);
            tiles += loss_tiles(end, rest);
            most = std::max(most, end.partial_bytes);
        }
        l.part = static_cast<float2 *>(c.take(8 * T * tiles));
        l.zt = static_cast<float *>(c.take(4 * T));
        l.partials = c.take(most);
        return l;
    }
    const int64_t tp = round_up(T, 256), vc = piece_columns(T, V);
    l.range_part = static_cast<float *>(c.take(4 * 3 * kRangeBlocks));
    l.ranges = static_cast<Ranges *>(c.take(sizeof(Ranges)));
    l.xt = static_cast<uint16_t *>(c.take(2 * K * tp));
    l.wt = static_cast<uint16_t *>(c.take(2 * K * vc));
    l.g = static_cast<uint16_t *>(c.take(2 * tp * vc));
    l.gt = static_cast<uint16_t *>(c.take(2 * tp * vc));
    l.dx = static_cast<float *>(c.take(4 * T * round_up(K, 4)));
    size_t most = 0;
    const int64_t rest = V % vc ? V % vc : vc;
    for (const int64_t cols : {vc < V ? vc : V, rest}) {
        const PiecePlans plans = plans_of(T, K, cols);
        most = std::max(most, std::max(plans.g.partial_bytes, std::max(plans.dx.partial_bytes, plans.dw.partial_bytes)));
        if (rest == cols) break;
    }
    l.partials = c.take(most);
    return l;
}

hipError_t pad16(const void *in, int64_t ld_in, int64_t rows, int64_t cols, uint16_t *out, int64_t ld_out, hipStream_t stream)
{
    const int64_t blocks = (rows * ld_out + 255) / 256;
    return launch(pad16_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, stream,
                  static_cast<const uint16_t *>(in), ld_in, rows, cols, out, ld_out);
}

// X and W as operands of the logits' product (padded copies in ws where needed)
hipError_t logits_operands(const XentProblem &p, const Layout &l, Operands &op, hipStream_t stream)
{
    const int64_t kp = round_up(p.K, 64);
    op.nk = (int)(kp / 64);
    op.M = (int)p.T;
    op.a = static_cast<const uint8_t *>(p.x);
    op.lda = 2 * p.ldx;
    op.b = static_cast<const uint8_t *>(p.w);
    op.ldb = 2 * p.ldw;
    if (p.K % 64 != 0) {
        if (hipError_t e = pad16(p.x, p.ldx, p.T, p.K, l.xp, kp, stream)) return e;
        if (hipError_t e = pad16(p.w, p.ldw, p.V, p.K, l.wp, kp, stream)) return e;
        op.a = reinterpret_cast<const uint8_t *>(l.xp);
        op.b = reinterpret_cast<const uint8_t *>(l.wp);
        op.lda = op.ldb = 2 * kp;
    }
    return hipSuccess;
}

}  // namespace

size_t xent_forward_workspace_bytes(int64_t T, int64_t K, int64_t V)
{
    Carve c{nullptr};
    carve(c, T, K, V, false);
    return c.at;
}
size_t xent_backward_workspace_bytes(int64_t T, int64_t K, int64_t V)
{
    Carve c{nullptr};
    carve(c, T, K, V, true);
    return c.at;
}

// the transposing copies' 128 x 128 tiles, of 256 threads; the products have fewer than half as many
bool xent_backward_fits_grid(int64_t T, int64_t K, int64_t V)
{
    const int64_t down = round_up(T, 256) / 128 + round_up(piece_columns(T, V), 128) / 128;
    return down * ((K + 127) / 128) <= kMaxItems / 256;
}

hipError_t launch_xent_forward(const XentProblem &p, void *ws, float *loss, float *lse, hipStream_t stream)
{
    Carve c{static_cast<uint8_t *>(ws)};
    const Layout l = carve(c, p.T, p.K, p.V, false);
    Operands lo{};
    if (hipError_t e = logits_operands(p, l, lo, stream)) return e;
    const int64_t step = loss_columns(p.T, p.V);
    int64_t tiles = 0;
    for (int64_t v0 = 0; v0 < p.V; v0 += step) {
        const int64_t cols = p.V - v0 < step ? p.V - v0 : step;
        Operands op = lo;
        op.b = lo.b + v0 * lo.ldb;
        op.N = (int)cols;
        const Plan plan = loss_plan(p.T, p.K, cols);
        const StatsEpi epi{l.part + tiles * p.T, l.zt, p.target, v0};
        if (hipError_t e = launch_product<BF16>(op, epi, plan, l.partials, stream)) return e;
        tiles += loss_tiles(plan, cols);
    }
    return launch(xent_join_kernel, dim3((unsigned)((p.T + 31) / 32)), dim3(256), 0, stream, l.part, (int)tiles, (int)p.T, p.V,
                  l.zt, p.target, p.ignore_index, loss, lse);
}

hipError_t launch_xent_backward(const XentProblem &p, const float *dloss, const float *dlse, const float *lse, void *ws,
                                void *dx, bool dx_bf16, void *dw, bool dw_bf16, hipStream_t stream)
{
    Carve c{static_cast<uint8_t *>(ws)};
    const Layout l = carve(c, p.T, p.K, p.V, true);
    const int64_t tp = round_up(p.T, 256), vc = piece_columns(p.T, p.V);
    Operands lo{};
    if (hipError_t e = logits_operands(p, l, lo, stream)) return e;
    const RowWeights weights{dloss, dlse, p.target, p.ignore_index, p.V};
    const bool vec = p.K % 8 == 0 && p.ldx % 8 == 0 && p.ldw % 8 == 0 && (uintptr_t)p.x % 16 == 0 && (uintptr_t)p.w % 16 == 0;
    const int64_t work = (p.T + p.V) * p.K;
    const int blocks = (int)(work > 8192 * kRangeBlocks ? kRangeBlocks : work / 8192 + 1);
    if (hipError_t e = launch(range_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, static_cast<const uint16_t *>(p.x), p.ldx,
                              static_cast<const uint16_t *>(p.w), p.ldw, p.T, p.K, p.V, vec ? 1 : 0, weights, l.range_part))
        return e;
    const int64_t ld_acc = round_up(p.K, 4);
    for (int64_t v0 = 0; v0 < p.V; v0 += vc) {
        const int64_t cols = p.V - v0 < vc ? p.V - v0 : vc;
        const bool first = v0 == 0, last = v0 + vc >= p.V;
        Operands op = lo;
        op.b = lo.b + v0 * lo.ldb;
        op.N = (int)cols;
        const GradEpi epi{weights, lse, v0, l.ranges, l.g, l.gt, vc, tp};
        const PiecePlans plans = plans_of(p.T, p.K, cols);
        const int64_t cols_done = plans.cols_done, rows_done = plans.rows_done;
        Turn tx{}, tw{};
        if (dw && first) tx = turn_of(p.x, p.ldx, p.T, p.K, l.xt, tp, tp);
        if (dx) tw = turn_of(static_cast<const uint16_t *>(p.w) + v0 * p.ldw, p.ldw, cols, p.K, l.wt, vc, cols_done);
        if (tx.tiles + tw.tiles > 0)
            if (hipError_t e = launch(turn_kernel, dim3((unsigned)(tx.tiles + tw.tiles)), dim3(256), 0, stream, tx, tw, weights,
                                      l.range_part, first ? blocks : 0, l.ranges))
                return e;
        if (hipError_t e = launch_product<BF16>(op, epi, plans.g, l.partials, stream)) return e;
        if (dx) {
            Operands q{};
            q.a = reinterpret_cast<const uint8_t *>(l.g);
            q.lda = 2 * vc;
            q.b = reinterpret_cast<const uint8_t *>(l.wt);
            q.ldb = 2 * vc;
            q.M = (int)p.T;
            q.N = (int)p.K;
            q.nk = (int)(cols_done / 64);
            auto run = [&](const auto &e) { return launch_product<F16>(q, e, plans.dx, l.partials, stream); };
            const float *add = first ? nullptr : l.dx;
            hipError_t e;
            if (!last)
                e = run(StoreEpi<false>{l.dx, ld_acc, 0, 1.0f, 0.0f, add, ld_acc, &l.ranges->up_gw});
            else if (dx_bf16)
                e = run(StoreEpi<true>{dx, p.K, 0, 1.0f, 0.0f, add, ld_acc, &l.ranges->up_gw});
            else
                e = run(StoreEpi<false>{dx, p.K, 0, 1.0f, 0.0f, add, ld_acc, &l.ranges->up_gw});
            if (e) return e;
        }
        if (dw) {
            Operands q{};
            q.a = reinterpret_cast<const uint8_t *>(l.gt);
            q.lda = 2 * tp;
            q.b = reinterpret_cast<const uint8_t *>(l.xt);
            q.ldb = 2 * tp;
            q.M = (int)cols;
            q.N = (int)p.K;
            q.nk = (int)(rows_done / 64);
            auto run = [&](const auto &e) { return launch_product<F16>(q, e, plans.dw, l.partials, stream); };
            const hipError_t e =
                dw_bf16 ? run(StoreEpi<true>{static_cast<uint16_t *>(dw) + v0 * p.K, p.K, 0, 1.0f, 0.0f, nullptr, 0, &l.ranges->up_gx})
                        : run(StoreEpi<false>{static_cast<float *>(dw) + v0 * p.K, p.K, 0, 1.0f, 0.0f, nullptr, 0, &l.ranges->up_gx});
            if (e) return e;
        }
    }
    return hipSuccess;
}

}  // namespace mx
