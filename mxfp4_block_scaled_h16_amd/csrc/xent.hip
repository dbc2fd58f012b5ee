// Softmax cross entropy of a linear head, in pieces of the vocabulary, without keeping the logits.
//
//   z = X W^T,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,target
//   G_tv = exp(z_tv - lse_t) (dloss_t + dlse_t) - [v = target_t] dloss_t,  dX = G W,  dW = G^T X
//
// Forward: one product whose epilogue leaves a maximum and a sum of exponentials per row and
// column tile, and a kernel that joins them. Backward: for each piece of the vocabulary the logits
// are formed again and leave the product's epilogue as G, in bf16 and in both orientations; dX
// adds up over the pieces in FP32, dW's rows of the piece are written once.
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
// (statistics in base 2, times log2 e), and the target's z where the tile holds it. A lane holds 32
// columns of a row per 32-row tile, its partner in the other half-wave the other 32 of the
// wavefront's 64; the wavefronts of a row join through the LDS.
struct StatsEpi {
    static constexpr bool kSym = false;
    float2 *part;            // [tiles_n][T]
    float *zt;               // [T]
    const int64_t *target;

    template <class G>
    __device__ __forceinline__ void run(v16f (&acc)[G::FI][G::FJ], const Where &w, const Operands &op, uint8_t *lds) const
    {
        const int r = w.lane & 31, half = w.lane >> 5;
        float2 *slots = reinterpret_cast<float2 *>(lds);   // [wave column][row of the tile]
        const int wn = w.wave / G::kWavesM;
        const int nleft = op.N - (w.n0 + w.col0 + 4 * half);   // valid: 32 j + 8 q + t < nleft
#pragma unroll
        for (int i = 0; i < G::FI; ++i) {
            const int row = w.row0 + 32 * i + r;
            const int m = min(w.m0 + row, op.M - 1);
            // the target's place among this lane's columns; far outside when it is not an index
            const int64_t tc = target[m] - (w.n0 + w.col0 + 4 * half);
            const int want = tc >= 0 && tc < 64 ? (int)tc : -1;
            float top = -INFINITY;
            float hit = 0.0f;
            bool found = false;
#pragma unroll
            for (int j = 0; j < G::FJ; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int c = 32 * j + 8 * (e / 4) + (e % 4);
                    float z = acc[i][j][e];
                    if (c == want) {
                        hit = z;
                        found = true;
                    }
                    z = c < nleft ? z * kLog2e : -INFINITY;
                    acc[i][j][e] = z;
                    top = fmaxf(top, z);
                }
            if (found && w.m0 + row < op.M && want < nleft) zt[m] = hit;
            top = fmaxf(top, __shfl_xor(top, 32));
            const float ref = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < G::FJ; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) sum += fast_exp2(acc[i][j][e] - ref);
            sum += __shfl_xor(sum, 32);
            if (half == 0) slots[wn * G::kTileM + row] = make_float2(top, sum);
        }
        __syncthreads();
        for (int row = threadIdx.x; row < G::kTileM; row += 64 * G::NW) {
            float2 s = slots[row];
#pragma unroll
            for (int k = 1; k < G::kWavesN; ++k) {
                const float2 o = slots[k * G::kTileM + row];
                const float top = fmaxf(s.x, o.x), ref = top == -INFINITY ? 0.0f : top;
                s = make_float2(top, s.y * fast_exp2(s.x - ref) + o.y * fast_exp2(o.x - ref));
            }
            const int m = w.m0 + row;
            if (m < op.M) part[(int64_t)(w.n0 / G::kTileN) * op.M + m] = s;
        }
    }
};

// Joins the column tiles of 32 rows: 8 threads per row, each every eighth tile.
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
        return make_float2(top, s.y * fast_exp2(s.x - ref) + o.y * fast_exp2(o.x - ref));
    };
    float2 s = make_float2(-INFINITY, 0.0f);
    if (t < T)
        for (int k = slice; k < tiles; k += 8) s = join(s, part[(int64_t)k * T + t]);
    slots[slice][lr] = s;
    __syncthreads();
    if (slice != 0 || t >= T) return;
    for (int k = 1; k < 8; ++k) s = join(s, slots[k][lr]);
    const float l = (s.x + log2f(s.y)) * kLn2;
    lse[t] = l;
    const int64_t tg = target[t];
    float v = 0.0f;
    if (tg != ignore_index) v = tg >= 0 && tg < V ? l - zt[t] : NAN;
    loss[t] = v;
}

// -------------------------------------------------------------------- the gradient's product --
// G of the tile in bf16 (one rounding: the products that read it take bf16), zero in rows past T, in
// columns past V and in rows whose target is ignored or no index (their dlse still counts: lse is
// an output of every row).
struct GradEpi {
    static constexpr bool kSym = false;
    const float *dloss, *dlse, *lse;
    const int64_t *target;
    int64_t ignore_index, V, v0;   // the piece's first column
    uint16_t *g, *gt;              // [Tp][ldg], [Vc][ldt]
    int64_t ldg, ldt;

    template <class G>
    __device__ __forceinline__ void run(v16f (&acc)[G::FI][G::FJ], const Where &w, const Operands &op, uint8_t *lds) const
    {
        const int r = w.lane & 31, half = w.lane >> 5;
        const int nbase = w.n0 + w.col0 + 4 * half;
        const int nleft = op.N - nbase;
#pragma unroll
        for (int i = 0; i < G::FI; ++i) {
            const int m = w.m0 + w.row0 + 32 * i + r;
            const bool live = m < op.M;
            const int mm = live ? m : op.M - 1;
            const int64_t tg = target[mm];
            const bool counts = live && tg != ignore_index && tg >= 0 && tg < V;
            const float dl = counts && dloss ? dloss[mm] : 0.0f;
            const float dp = dl + (live && dlse ? dlse[mm] : 0.0f);
            const float ref = lse[mm] * kLog2e;
            const int64_t tc = tg - v0 - nbase;
            const int want = counts && tc >= 0 && tc < 64 ? (int)tc : -1;
#pragma unroll
            for (int j = 0; j < G::FJ; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int c = 32 * j + 8 * (e / 4) + (e % 4);
                    float v = fast_exp2(fmaf(acc[i][j][e], kLog2e, -ref)) * dp;
                    if (c == want) v -= dl;
                    // dp == 0: the row's gradient is zero whatever its logits are
                    acc[i][j][e] = c < nleft && dp != 0.0f ? v : (c == want ? -dl : 0.0f);
                }
        }
        store_tile16<G>(w, lds, [](float a, float b) { return pack_bf16(a, b); },
                        [&](int i, int j, int q) {
                            return f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                        },
                        g, ldg, gt, ldt);
    }
};

// ------------------------------------------------------------------------------- copies -------
// Which rows of X add something to the gradients: the others are taken as zeros in the transposed
// copy, so that what a padded position holds (a NaN) meets no zero of G.
struct RowWeights {
    const float *dloss, *dlse;   // NULL: zeros
    const int64_t *target;       // NULL: every row counts
    int64_t ignore_index, V;
    __device__ __forceinline__ bool live(int64_t t) const
    {
        if (!target) return true;
        const int64_t tg = target[t];
        return (dlse && dlse[t] != 0.0f) || (dloss && tg != ignore_index && tg >= 0 && tg < V && dloss[t] != 0.0f);
    }
};

// out[c][r] = in[r][c] (16-bit), r < rows, c < cols; zero for rows <= r < rows_padded
__global__ __launch_bounds__(256) void transpose16_kernel(const uint16_t *__restrict__ in, int64_t ld_in, int64_t rows,
                                                          int64_t cols, uint16_t *__restrict__ out, int64_t ld_out,
                                                          int64_t rows_padded, RowWeights weights)
{
    __shared__ uint16_t tile[64][64 + 2];
    const int64_t r0 = (int64_t)blockIdx.x * 64, c0 = (int64_t)blockIdx.y * 64;
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int64_t r = r0 + ty + 4 * k, c = c0 + tx;
        tile[ty + 4 * k][tx] = r < rows && c < cols && weights.live(r) ? in[r * ld_in + c] : (uint16_t)0;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int64_t c = c0 + ty + 4 * k, r = r0 + tx;
        if (c < cols && r < rows_padded) out[c * ld_out + r] = tile[tx][ty + 4 * k];
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

hipError_t transpose16(const void *in, int64_t ld_in, int64_t rows, int64_t cols, uint16_t *out, int64_t ld_out,
                       int64_t rows_padded, const RowWeights &weights, hipStream_t stream)
{
    return launch(transpose16_kernel, dim3((unsigned)((rows_padded + 63) / 64), (unsigned)((cols + 63) / 64)), dim3(256), 0,
                  stream, static_cast<const uint16_t *>(in), ld_in, rows, cols, out, ld_out, rows_padded, weights);
}

// ------------------------------------------------------------------------------ workspace -----
// tiles of 256 x 256 where there are enough of them, else of 128 x 128
bool big_tiles(int64_t M, int64_t N) { return ((M + 255) / 256) * ((N + 255) / 256) > kComputeUnits / 2; }

// Pieces of the vocabulary: G takes at most 256 MB per orientation, so that a piece stays near the
// last-level cache, and a piece has at least 2048 columns.
int64_t piece_columns(int64_t T, int64_t V)
{
    const int64_t tp = round_up(T, 256);
    int64_t most = ((int64_t)1 << 27) / tp / 256 * 256;
    if (most < 2048) most = 2048;
    const int64_t pieces = (V + most - 1) / most;
    return round_up((V + pieces - 1) / pieces, 256);
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
    uint16_t *xp, *wp;   // copies of X and W with rows padded to whole stages (K % 32 != 0)
    float2 *part;
    float *zt;
    uint16_t *xt, *wt, *g, *gt;
    float *dx;
};
Layout carve(Carve &c, int64_t T, int64_t K, int64_t V, bool backward)
{
    Layout l{};
    const int64_t kp = round_up(K, 32);
    if (K % 32 != 0) {
        l.xp = static_cast<uint16_t *>(c.take(2 * T * kp));
        l.wp = static_cast<uint16_t *>(c.take(2 * V * kp));
    }
    if (!backward) {
        l.part = static_cast<float2 *>(c.take(8 * T * ((V + 127) / 128)));
        l.zt = static_cast<float *>(c.take(4 * T));
        return l;
    }
    const int64_t tp = round_up(T, 256), vc = piece_columns(T, V);
    l.xt = static_cast<uint16_t *>(c.take(2 * K * tp));
    l.wt = static_cast<uint16_t *>(c.take(2 * K * vc));
    l.g = static_cast<uint16_t *>(c.take(2 * tp * vc));
    l.gt = static_cast<uint16_t *>(c.take(2 * tp * vc));
    l.dx = static_cast<float *>(c.take(4 * T * round_up(K, 4)));
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
    const int64_t kp = round_up(p.K, 32);
    op.nk = (int)(kp / 32);
    op.M = (int)p.T;
    op.a = static_cast<const uint8_t *>(p.x);
    op.lda = 2 * p.ldx;
    op.b = static_cast<const uint8_t *>(p.w);
    op.ldb = 2 * p.ldw;
    if (p.K % 32 != 0) {
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

hipError_t launch_xent_forward(const XentProblem &p, void *ws, float *loss, float *lse, hipStream_t stream)
{
    Carve c{static_cast<uint8_t *>(ws)};
    const Layout l = carve(c, p.T, p.K, p.V, false);
    Operands op{};
    if (hipError_t e = logits_operands(p, l, op, stream)) return e;
    op.N = (int)p.V;
    const StatsEpi epi{l.part, l.zt, p.target};
    const bool big = big_tiles(p.T, p.V);
    if (hipError_t e = big ? launch_product<BF16, Big>(op, epi, 1, stream) : launch_product<BF16, Small>(op, epi, 1, stream))
        return e;
    const int tiles = (int)((p.V + (big ? 255 : 127)) / (big ? 256 : 128));
    return launch(xent_join_kernel, dim3((unsigned)((p.T + 31) / 32)), dim3(256), 0, stream, l.part, tiles, (int)p.T, p.V,
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
    if (dw)
        if (hipError_t e = transpose16(p.x, p.ldx, p.T, p.K, l.xt, tp, tp,
                                       RowWeights{dloss, dlse, p.target, p.ignore_index, p.V}, stream))
            return e;
    const int64_t ld_acc = round_up(p.K, 4);
    for (int64_t v0 = 0; v0 < p.V; v0 += vc) {
        const int64_t cols = p.V - v0 < vc ? p.V - v0 : vc;
        const bool first = v0 == 0, last = v0 + vc >= p.V;
        Operands op = lo;
        op.b = lo.b + v0 * lo.ldb;
        op.N = (int)cols;
        const GradEpi epi{dloss, dlse, lse, p.target, p.ignore_index, p.V, v0, l.g, l.gt, vc, tp};
        const bool big = big_tiles(p.T, cols);
        if (hipError_t e = big ? launch_product<BF16, Big>(op, epi, 1, stream) : launch_product<BF16, Small>(op, epi, 1, stream))
            return e;
        // G covers whole tiles; the products over it run to the end of the last one
        const int64_t step = big ? 256 : 128;
        const int64_t cols_done = round_up(cols, step), rows_done = round_up(p.T, step);
        if (dx) {
            if (hipError_t e = transpose16(static_cast<const uint16_t *>(p.w) + v0 * p.ldw, p.ldw, cols, p.K, l.wt, vc,
                                           cols_done, RowWeights{}, stream))
                return e;
            Operands q{};
            q.a = reinterpret_cast<const uint8_t *>(l.g);
            q.lda = 2 * vc;
            q.b = reinterpret_cast<const uint8_t *>(l.wt);
            q.ldb = 2 * vc;
            q.M = (int)p.T;
            q.N = (int)p.K;
            q.nk = (int)(cols_done / 32);
            auto run = [&](const auto &e) {
                return big_tiles(p.T, p.K) ? launch_product<BF16, Big>(q, e, 1, stream)
                                           : launch_product<BF16, Small>(q, e, 1, stream);
            };
            const float *add = first ? nullptr : l.dx;
            hipError_t e;
            if (!last)
                e = run(StoreEpi<false>{l.dx, ld_acc, 0, 1.0f, 0.0f, add, ld_acc});
            else if (dx_bf16)
                e = run(StoreEpi<true>{dx, p.K, 0, 1.0f, 0.0f, add, ld_acc});
            else
                e = run(StoreEpi<false>{dx, p.K, 0, 1.0f, 0.0f, add, ld_acc});
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
            q.nk = (int)(rows_done / 32);
            auto run = [&](const auto &e) {
                return big_tiles(cols, p.K) ? launch_product<BF16, Big>(q, e, 1, stream)
                                            : launch_product<BF16, Small>(q, e, 1, stream);
            };
            const hipError_t e =
                dw_bf16 ? run(StoreEpi<true>{static_cast<uint16_t *>(dw) + v0 * p.K, p.K, 0, 1.0f, 0.0f})
                        : run(StoreEpi<false>{static_cast<float *>(dw) + v0 * p.K, p.K, 0, 1.0f, 0.0f});
            if (e) return e;
        }
    }
    return hipSuccess;
}

}  // namespace mx
