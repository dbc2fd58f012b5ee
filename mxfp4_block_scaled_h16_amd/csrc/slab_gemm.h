// Matrix products C[m][n] = sum_k A[m][k] B[n][k] on gfx950's matrix cores, for 8- and 16-bit
// elements and with an epilogue of the caller's (device code, header only).
//
// Both operands are row-major along k. A stage is 128 bytes of every row of the workgroup's tile
// (64 values of 16 bits, 128 of 8 bits: a whole cache line, and with 8 bits a whole scale block),
// brought from memory to the LDS by direct 16-byte-per-lane loads into two stage buffers. In
// units of 128-byte rows every element type costs the same: per stage and 16 x 16 output tile two
// v_mfma_f32_16x16x32 (16-bit) or one v_mfma_scale_f32_16x16x128_f8f6f4 (8-bit), 32 matrix-core
// cycles either way, so one tiling and one pipeline serve them all.
//
// Measured at 8192 x 8192 x 8192 in bf16 (TFLOP/s in turn on one card): stages of 64 bytes in a ring
// of four, which ask the L1 for every line twice: 1213; of 128 bytes: 1348; with buffer loads, whose
// addresses are one register and a scalar: 1390. 32 x 32 MFMAs instead of 16 x 16: 1274. Loads spread
// over the second half of a stage instead of bunched behind the barrier: 1360; a second barrier
// that leaves them half a stage longer: 1340.
//
// In FP8 a stage takes as long, for twice the values: 8192 x 6144 x 4096 174 to 215 us by the power that the card
// has left, 187 on average, 2.2 PFLOP/s (the library with one scale for each matrix, in turn with it: 142 to 177, 154);
// 4096 x 14336 x 8192 376 us, 2.56 PFLOP/s (316). What is left is the power cap and the epilogue, which the next tile does not
// overlap. A workgroup per CU that walks over its tiles with the next tile's loads ahead of the epilogue needs
// registers that are not there (9 to 28 spilled) and was slower: FP16 896 tiles 17%, bf16 heads 2%.
//
// The rows of a stage buffer hold their eight 16-byte chunks XOR-permuted by bits 1-3 of the row: the
// 16 lanes that the LDS serves at a time read one chunk of 16 rows, and so 16 distinct bank groups.
//
// The product is formed transposed (B as the first operand of the MFMA), so a lane ends with
// one row of C per 16-row tile and runs of four consecutive columns: register t of acc[i][j] in lane
// (r, q), r = lane % 16, q = lane / 16, is C[m0 + row0 + 16 i + r][n0 + col0 + 16 j + 4 q + t].
// Row statistics (a softmax) then need two cross-lane steps, and the output goes through the LDS
// so that stores cover whole lines.
#pragma once

#include <climits>
#include <utility>

#include "internal.h"
#include "train_internal.h"

namespace mx {
namespace slab {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void_t;
typedef const __attribute__((address_space(1))) void gbl_void_t;

constexpr int kRowBytes = 128;   // bytes of a row per stage
constexpr int kRowsPerDma = 8;   // a wave-wide 16-byte-per-lane load covers 8 rows of a stage
constexpr int kComputeUnits = 256;

// ------------------------------------------------------------------------- element types ------
struct BF16 {
    static constexpr bool kScaled = false;
    static __device__ __forceinline__ void mfma(f32x4 &acc, const u32x4 &b, const u32x4 &a)
    {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a),
                                                      acc, 0, 0, 0);
    }
};
struct F16 {
    static constexpr bool kScaled = false;
    static __device__ __forceinline__ void mfma(f32x4 &acc, const u32x4 &b, const u32x4 &a)
    {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a),
                                                     acc, 0, 0, 0);
    }
};
// E4M3 codes with an E8M0 scale byte for each 128 values of a row. A lane supplies 32 of the 128
// values of a stage; which 32 does not matter, as A and B take the same ones and all share a scale.
struct E4M3 {
    static constexpr bool kScaled = true;
    // the scales are bytes BB of sb and BA of sa
    template <int BB, int BA>
    static __device__ __forceinline__ void mfma(f32x4 &acc, const u32x4 &b0, const u32x4 &b1, const u32x4 &a0,
                                                const u32x4 &a1, uint32_t sb, uint32_t sa)
    {
        const v8i vb = {(int)b0.x, (int)b0.y, (int)b0.z, (int)b0.w, (int)b1.x, (int)b1.y, (int)b1.z, (int)b1.w};
        const v8i va = {(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vb, va, acc, 0, 0, BB, (int)sb, BA, (int)sa);
    }
};

// s_waitcnt vmcnt(N) (gfx9 encoding; the other counters at their no-wait maxima)
template <int N>
__device__ __forceinline__ void wait_vmcnt()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

__device__ __forceinline__ void barrier()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

// Between LDS accesses by which lanes of one wavefront hand values to each other: its LDS instructions are carried out in
// their order, so it is the compiler alone that must not move one across; no instruction comes of it.
__device__ __forceinline__ void lds_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
}

// f(0), f(1), ... f(N - 1), the numbers as types
template <class F, int... K>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, K...>)
{
    (f(std::integral_constant<int, K>()), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F f)
{
    each_of(f, std::make_integer_sequence<int, N>());
}

__device__ __forceinline__ int chunk_perm(int row) { return (row >> 1) & 7; }

// ------------------------------------------------------------------------------ geometry ------
// NW_ wavefronts on a TM x TN tile, arranged WM x (NW_ / WM); NB stage buffers.
template <int NW_, int TM, int TN, int WM, int NB = 2>
struct Geo {
    static constexpr int NW = NW_, kTileM = TM, kTileN = TN, kBuffers = NB;
    static_assert(NB == 2 || NB == 4, "the buffer of a stage is its low bits");
    static constexpr int kABytes = TM * kRowBytes;
    static constexpr int kStageBytes = (TM + TN) * kRowBytes;
    static constexpr int kRingBytes = NB * kStageBytes;
    static constexpr int kScaleSlot = (TM + TN) * 16;             // 16 scale bytes per row: 16 stages
    static constexpr int kWavesM = WM, kWavesN = NW / WM;
    static constexpr int kWaveRows = TM / kWavesM, kWaveCols = TN / kWavesN;
    static constexpr int FI = kWaveRows / 16, FJ = kWaveCols / 16;
    static constexpr int kDmaA = TM / kRowsPerDma / NW, kDmaB = TN / kRowsPerDma / NW;
    static constexpr int kDmaPerStage = kDmaA + kDmaB;
    static_assert(kDmaA * kRowsPerDma * NW == TM && kDmaB * kRowsPerDma * NW == TN, "whole loads per wavefront");
    static_assert(TM + TN <= 64 * NW, "a thread for each row's scales");
    // a wavefront's part of the LDS in the epilogue, 32 rows of its tile in FP32: one stage buffer in all
    static constexpr int kBlockRows = 32, kEpiBlocks = kWaveRows / kBlockRows;
    static constexpr int kEpiWave = kBlockRows * kWaveCols * 4;
    static_assert(NW * kEpiWave <= kStageBytes, "the epilogue works in a stage buffer");
    // behind the stage buffers: scales, or 16 bytes for each row of the tile for the epilogue's use
    template <class E>
    static constexpr int lds_bytes()
    {
        return kRingBytes + (E::kScaled ? 2 * kScaleSlot : TM * 16);
    }
    static constexpr int kMinBlocks = kRingBytes + 2 * kScaleSlot <= 80 * 1024 ? 2 : 1;   // workgroups per CU
};
using Big = Geo<8, 256, 256, 2>;       // wave tiles 128 x 64, 128 accumulator registers
using Small = Geo<4, 128, 128, 2>;     // wave tiles 64 x 64, two workgroups per CU
using Tiny = Geo<4, 64, 64, 2, 4>;     // wave tiles 32 x 32, loads three stages ahead: where latency is all

// --------------------------------------------------------------------------------- operands ---
// Rows past M and N are read as row M - 1 and N - 1 (their results are the epilogue's to drop).
// Every row is readable, and zero past its length, up to nk whole stages; 16-byte aligned.
struct Operands {
    const uint8_t *a, *b;
    int64_t lda, ldb;          // bytes
    const uint8_t *as, *bs;    // E4M3: scale rows, 16-byte aligned, readable in whole 16 bytes
    int64_t ldas, ldbs;
    int M, N, nk;
    int tiles_m, tiles_n;
    int64_t batch_a, batch_b;  // bytes from one product of a batch to the next
    // The first `whole` tiles of all products have a workgroup each. The others, which would leave much of the chip
    // idle, are worked by `splits` workgroups each, stages [y per, y per + per) by the y-th: these leave their
    // sums in partials, in the order of their registers, and finish_kernel adds them up.
    int whole, splits, per;
    f32x4 *partials;
};

struct Where {
    int m0, n0;      // tile origin
    int wave, lane;
    int row0, col0;  // the wavefront's origin in the tile
    int batch;
    int block0, block1;   // the blocks of 32 rows of every wavefront that the epilogue is for
};

// Where workgroup v of n neighbours works in their order: consecutive workgroups go to the eight XCDs in
// turn; each XCD gets a contiguous range.
__device__ __forceinline__ int spread(int v, int n)
{
    const int per = n / 8, rem = n % 8, x = v % 8;
    return x * per + min(x, rem) + v / 8;
}

// Tile t of a product. Tiles are walked column by column in groups of row panels covering 1024 rows, so that
// the workgroups running on one XCD share operand panels in its L2. SYM: only the tiles that touch
// the lower triangle of a square of tiles, in bands of four rows of tiles, each in squares of 4 x 4 and
// what is left at the diagonal.
template <class G, bool SYM>
__device__ __forceinline__ void locate(int t, int tiles_m, int tiles_n, int &m0, int &n0)
{
    if constexpr (SYM) {
        // band I holds 16 I + 10 tiles, the bands before it 8 I I + 2 I (a short last band fewer)
        int band = (int)sqrtf((float)t * 0.125f);   // a start that the loops put right
        while (8 * band * band + 2 * band > t) --band;
        while (8 * (band + 1) * (band + 1) + 2 * (band + 1) <= t && 4 * (band + 1) < tiles_m) ++band;
        const int in = t - (8 * band * band + 2 * band), high = min(4, tiles_m - 4 * band), square = 4 * high;
        int i, j;
        if (in < band * square) {
            i = in % square % high;
            j = in / square * 4 + in % square / high;
        } else {
            int rest = in - band * square;
            for (i = 0; rest > i; ++i) rest -= i + 1;
            j = 4 * band + rest;
        }
        m0 = (4 * band + i) * G::kTileM;
        n0 = j * G::kTileN;
    } else {
        constexpr int kGroupRows = 1024 / G::kTileM;
        const int group = kGroupRows * tiles_n;
        const int g0 = (t / group) * kGroupRows;
        const int gm = min(kGroupRows, tiles_m - g0);
        m0 = (g0 + (t % group) % gm) * G::kTileM;
        n0 = ((t % group) / gm) * G::kTileN;
    }
}

// where split y of the i-th split tile keeps its sums
template <class G>
__device__ __forceinline__ f32x4 *partial_at(const Operands &op, int i, int y)
{
    return op.partials + ((int64_t)i * op.splits + y) * (G::kTileM * G::kTileN / 4);
}

// tile t of all products: its batch and origin
template <class G, class Epi>
__device__ __forceinline__ void place(Where &w, const Operands &op, int t)
{
    const int tiles = Epi::kSym ? op.tiles_m * (op.tiles_m + 1) / 2 : op.tiles_m * op.tiles_n;
    w.batch = t < tiles ? 0 : t / tiles;
    locate<G, Epi::kSym>(t - w.batch * tiles, op.tiles_m, op.tiles_n, w.m0, w.n0);
    w.lane = threadIdx.x & 63;
    w.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    w.row0 = w.wave % G::kWavesM * G::kWaveRows;
    w.col0 = w.wave / G::kWavesM * G::kWaveCols;
    w.block0 = 0;
    w.block1 = G::kEpiBlocks;
}

// -------------------------------------------------------------------------------- the kernel --
// Epi: a trivially copyable functor with kSym and
//   template <class G> __device__ void run(f32x4 (&acc)[FI][FJ], const Where &, const Operands &, uint8_t *lds, uint8_t *info)
// called by every wavefront with a stage buffer that nothing else uses (lds) and, for 16-bit operands, 16 bytes
// of LDS for each row of the tile (info).
//
// A stage is worked in two halves of its MFMAs. During the first, the fragments of the second are
// read from the LDS; then nothing of the stage is left to read, and one barrier says both that its
// buffer is free, for the loads of stage s + 2, and that stage s + 1 has landed, whose first
// fragments are read during the second half. (16-bit: the halves are those of the row's 128
// bytes. 8-bit: one MFMA takes a lane's part of all 128, so the halves are the upper and lower
// rows of the wavefront's tile, and B's fragments give way to the next stage's column by column.)
template <class E, class G, class Epi>
__global__ __launch_bounds__(64 * G::NW, G::kMinBlocks) void product_kernel(Operands op, Epi epi)
{
#if defined(__HIP_DEVICE_COMPILE__)   // the buffer-resource builtins do not exist in the host's pass
    constexpr int FI = G::FI, FJ = G::FJ, NB = G::kBuffers;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[G::template lds_bytes<E>()];

    // this workgroup's tile and stages
    Where w;
    int first = 0, end = op.nk, split_tile = -1, split = 0;
    const int tile = blockIdx.x;
    if (tile < op.whole) {
        place<G, Epi>(w, op, spread(tile, op.whole));
    } else {
        const int rest = (int)gridDim.x - op.whole, tail = rest / op.splits;
        const int i = spread(tile - op.whole, rest);
        split = i / tail;
        split_tile = i - split * tail;
        place<G, Epi>(w, op, op.whole + split_tile);
        first = split * op.per;
        end = min(op.nk, first + op.per);
    }
    const int lane = w.lane, r = lane & 15, q = lane >> 4;

    // load u of this wavefront fills rows [8 (kDma wave + u), + 8) of the stage: lane L the 16 bytes at
    // row L / 8, physical chunk L % 8, from the row's chunk (L % 8) ^ perm(row)
    const int a_row0 = kRowsPerDma * G::kDmaA * w.wave, b_row0 = kRowsPerDma * G::kDmaB * w.wave;
    const uint8_t *abase, *bbase;
    uint32_t aoff[G::kDmaA], boff[G::kDmaB];
    // E4M3: a thread per row of the tile (A's first, then B's) takes the scales of 16 stages, 16 bytes, and lays
    // them into one of two slots of the LDS: [stage][64 rows][row % 16][row / 16], so that a lane has the
    // scales of its row in four 16-row tiles in one word.
    const uint8_t *srow = nullptr;
    auto aim = [&](const Where &t) {   // the loads' addresses for tile t
        abase = op.a + t.batch * op.batch_a + (int64_t)t.m0 * op.lda;
        bbase = op.b + t.batch * op.batch_b + (int64_t)t.n0 * op.ldb;
#pragma unroll
        for (int u = 0; u < G::kDmaA; ++u) {
            const int row = a_row0 + kRowsPerDma * u + lane / 8;
            aoff[u] = (uint32_t)min(row, op.M - 1 - t.m0) * (uint32_t)op.lda + 16u * ((lane % 8) ^ chunk_perm(row));
        }
#pragma unroll
        for (int u = 0; u < G::kDmaB; ++u) {
            const int row = b_row0 + kRowsPerDma * u + lane / 8;
            boff[u] = (uint32_t)min(row, op.N - 1 - t.n0) * (uint32_t)op.ldb + 16u * ((lane % 8) ^ chunk_perm(row));
        }
    };
    auto aim_scales = [&](const Where &t) {
        const bool is_b = (int)threadIdx.x >= G::kTileM;
        const int row = min((int)threadIdx.x, G::kTileM + G::kTileN - 1) - (is_b ? G::kTileM : 0);
        srow = is_b ? op.bs + (int64_t)(t.n0 + min(row, op.N - 1 - t.n0)) * op.ldbs
                    : op.as + (int64_t)(t.m0 + min(row, op.M - 1 - t.m0)) * op.ldas;
    };
    aim(w);
    auto buffer = [&](int stage) { return lds + (stage & (NB - 1)) * G::kStageBytes; };
    auto dma = [&](int stage, uint8_t *dst) {
        const auto arsrc = __builtin_amdgcn_make_buffer_rsrc((void *)abase, 0, 0xFFFFFFFFu, 0x00027000);
        const auto brsrc = __builtin_amdgcn_make_buffer_rsrc((void *)bbase, 0, 0xFFFFFFFFu, 0x00027000);
        const int at = stage * kRowBytes;
#pragma unroll
        for (int u = 0; u < G::kDmaA; ++u)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(arsrc, (lds_void_t *)(dst + a_row0 * kRowBytes + u * 1024), 16, aoff[u],
                                                     at, 0, 0);
#pragma unroll
        for (int u = 0; u < G::kDmaB; ++u)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(brsrc, (lds_void_t *)(dst + G::kABytes + b_row0 * kRowBytes + u * 1024),
                                                     16, boff[u], at, 0, 0);
    };
    // the loads behind the barrier of stage s; past the last stage the last one again, into a free buffer, so that
    // every wait counts alike
    auto load_ahead = [&](int s) { dma(min(s + NB, end - 1), buffer(s + NB)); };
    const int last_group = (end - 1) / 16;
    auto load_scales = [&](int g) { return *reinterpret_cast<const u32x4 *>(srow + (int64_t)min(g, last_group) * 16); };
    auto put_scales = [&](int g, const u32x4 &v) {
        if (G::kTileM + G::kTileN < 64 * G::NW && (int)threadIdx.x >= G::kTileM + G::kTileN) return;
        const bool is_b = (int)threadIdx.x >= G::kTileM;
        const int row = (int)threadIdx.x - (is_b ? G::kTileM : 0);
        uint8_t *dst = lds + G::kRingBytes + (g & 1) * G::kScaleSlot + (is_b ? G::kTileM : 0) + row / 64 * 64 +
                       row % 16 * 4 + row % 64 / 16;
#pragma unroll
        for (int k = 0; k < 16; ++k) dst[k * (G::kTileM + G::kTileN)] = (uint8_t)(v[k / 4] >> (8 * (k % 4)));
    };

    const int perm = chunk_perm(r);
    const int a_frag = (w.row0 + r) * kRowBytes, b_frag = G::kABytes + (w.col0 + r) * kRowBytes;
    const int chunk0 = 16 * (q ^ perm), chunk1 = 16 * ((4 + q) ^ perm);
    auto read_a = [&](const uint8_t *src, int i) { return *reinterpret_cast<const u32x4 *>(src + a_frag + 16 * i * kRowBytes); };
    auto read_b = [&](const uint8_t *src, int j) { return *reinterpret_cast<const u32x4 *>(src + b_frag + 16 * j * kRowBytes); };

    f32x4 acc[FI][FJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) acc[i][j] = f32x4{};

    if constexpr (E::kScaled) {
        aim_scales(w);
        const u32x4 v0 = load_scales(first >> 4), v1 = load_scales((first >> 4) + 1);
        put_scales(first >> 4, v0);
        put_scales((first >> 4) + 1, v1);
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): for the barrier below
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) dma(min(first + k, end - 1), buffer(first + k));
    wait_vmcnt<(NB - 1) * G::kDmaPerStage>();
    barrier();

    // 16-bit: the fragments of a half stage, twice. 8-bit: of a stage, and its scales.
    u32x4 fa0[FI], fb0[FJ], fa1[FI], fb1[FJ];
    auto read = [&](const uint8_t *src, u32x4 (&fa)[FI], u32x4 (&fb)[FJ]) {
#pragma unroll
        for (int j = 0; j < FJ; ++j) fb[j] = read_b(src, j);
#pragma unroll
        for (int i = 0; i < FI; ++i) fa[i] = read_a(src, i);
    };
    constexpr int H = FI / 2, WA = (FI + 3) / 4, WB = (FJ + 3) / 4;
    static_assert(H <= FJ, "an upper row for each column");
    uint32_t sa[WA], sb[WB], ta[WA], tb[WB];
    u32x4 next_scales = {};
    auto take_scales = [&](int stage, int slot, uint32_t (&xa)[WA], uint32_t (&xb)[WB]) {
        // wave tiles of 32 rows start in the middle of a word
        const int a_shift = FI < 4 ? w.row0 % 64 / 2 : 0, b_shift = FJ < 4 ? w.col0 % 64 / 2 : 0;
        const uint8_t *src =
            lds + G::kRingBytes + (slot & 1) * G::kScaleSlot + (stage & 15) * (G::kTileM + G::kTileN) + 4 * r;
#pragma unroll
        for (int k = 0; k < WA; ++k)
            xa[k] = *reinterpret_cast<const uint32_t *>(src + w.row0 / 64 * 64 + 64 * k) >> a_shift;
#pragma unroll
        for (int k = 0; k < WB; ++k)
            xb[k] = *reinterpret_cast<const uint32_t *>(src + G::kTileM + w.col0 / 64 * 64 + 64 * k) >> b_shift;
    };
    auto take_a = [&](const uint8_t *src, int i) {
        fa0[i] = read_a(src + chunk0, i);
        fa1[i] = read_a(src + chunk1, i);
    };
    auto take_b = [&](const uint8_t *src, int j) {
        fb0[j] = read_b(src + chunk0, j);
        fb1[j] = read_b(src + chunk1, j);
    };
    // the tile's first fragments
    if constexpr (!E::kScaled) {
        read(buffer(first) + chunk0, fa0, fb0);
    } else {
#pragma unroll
        for (int j = 0; j < FJ; ++j) take_b(buffer(first), j);
#pragma unroll
        for (int i = 0; i < H; ++i) take_a(buffer(first), i);
        take_scales(first, first >> 4, sa, sb);
    }
    if constexpr (!E::kScaled) {
        auto mfmas = [&](const u32x4 (&fa)[FI], const u32x4 (&fb)[FJ]) {
#pragma unroll
            for (int i = 0; i < FI; ++i)
#pragma unroll
                for (int j = 0; j < FJ; ++j) E::mfma(acc[i][j], fb[j], fa[i]);
        };
        constexpr int kMfma = FI * FJ, kReads = FI + FJ, kLoads = G::kDmaPerStage;
        constexpr int kPer = kMfma / kReads;   // MFMAs per read in the first half
        for (int s = first; s < end; ++s) {
            read(buffer(s) + chunk1, fa1, fb1);
            mfmas(fa0, fb0);
            if constexpr (kPer > 0) {
#pragma unroll
                for (int k = 0; k < kReads; ++k) {
                    __builtin_amdgcn_sched_group_barrier(0x008, kPer, 0);  // MFMA
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);     // DS read
                }
                __builtin_amdgcn_sched_group_barrier(0x008, kMfma - kPer * kReads, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the stage has been read
            wait_vmcnt<(NB - 2) * G::kDmaPerStage>();   // stage s + 1 has landed
            barrier();
            // the loads at once: they have the longest way to go
            load_ahead(s);
            read(buffer(s + 1) + chunk0, fa0, fb0);
            mfmas(fa1, fb1);
            if constexpr (kLoads + kReads <= kMfma) {
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // VMEM read
                }
#pragma unroll
                for (int k = 0; k < kReads; ++k) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                }
                __builtin_amdgcn_sched_group_barrier(0x008, kMfma - kLoads - kReads, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    } else {
        auto mfma = [&](auto I, auto J) {
            constexpr int i = decltype(I)::value, j = decltype(J)::value;
            E::template mfma<j % 4, i % 4>(acc[i][j], fb0[j], fb1[j], fa0[i], fa1[i], sb[j / 4], sa[i / 4]);
        };
        for (int s = first; s < end; ++s) {
            // the upper rows; the lower rows' fragments are read behind each group of MFMAs
            const uint8_t *now = buffer(s), *then = buffer(s + 1);
            each<H>([&](auto I) {
                take_a(now, H + decltype(I)::value);
                each<FJ>([&](auto J) { mfma(I, J); });
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, FJ - 1, 0);
            });
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
            wait_vmcnt<(NB - 2) * G::kDmaPerStage>();
            barrier();
            // the next 16 stages' scales: asked for early in these 16, laid down in the middle of them (those of
            // a split that starts between the two are there already)
            if ((s & 15) == 2 && (s >> 4) < last_group) next_scales = load_scales((s >> 4) + 1);
            if ((s & 15) == 8 && (s >> 4) < last_group && s - 6 >= first) put_scales((s >> 4) + 1, next_scales);
            load_ahead(s);
            take_scales(s + 1, (s + 1) >> 4, ta, tb);
            // the lower rows column by column; column j's fragments and those of upper row j follow it
            each<FJ>([&](auto J) {
                constexpr int j = decltype(J)::value;
                each<H>([&](auto I) { mfma(std::integral_constant<int, H + decltype(I)::value>(), J); });
                __builtin_amdgcn_sched_barrier(0);
                take_b(then, j);
                if (j < H) take_a(then, j);
            });
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < WA; ++k) sa[k] = ta[k];
#pragma unroll
            for (int k = 0; k < WB; ++k) sb[k] = tb[k];
        }
    }
    // the last stage's buffer is the epilogue's: every load has landed and every wavefront is past its reads
    wait_vmcnt<0>();
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    barrier();
    if (split_tile >= 0) {
        f32x4 *out = partial_at<G>(op, split_tile, split) + threadIdx.x;
#pragma unroll
        for (int i = 0; i < FI; ++i)
#pragma unroll
            for (int j = 0; j < FJ; ++j) out[(i * FJ + j) * 64 * G::NW] = acc[i][j];
        return;
    }
    epi.template run<G>(acc, w, op, buffer(end - 1), lds + G::kRingBytes);
#endif
}

// The sums of a split contraction, in their order (so that the result does not depend on which workgroup
// came first), and the epilogue. A tile's blocks of 32 rows have a workgroup each: what bounds this kernel is
// how fast a CU reads (a 256 x 256 tile of nine splits by one workgroup: 39 us).
template <class G, class Epi>
__global__ __launch_bounds__(64 * G::NW, G::kMinBlocks) void finish_kernel(Operands op, Epi epi)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[G::kStageBytes + G::kTileM * 16];
    const int tile = blockIdx.x / G::kEpiBlocks, blk = blockIdx.x % G::kEpiBlocks;
    Where w;
    place<G, Epi>(w, op, op.whole + tile);
    w.block0 = blk;
    w.block1 = blk + 1;
    f32x4 sum[2][G::FJ];
    for (int y = 0; y < op.splits; ++y) {
        const f32x4 *in = partial_at<G>(op, tile, y) + threadIdx.x + 2 * blk * G::FJ * 64 * G::NW;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < G::FJ; ++j) {
                const f32x4 v = in[(i * G::FJ + j) * 64 * G::NW];
                sum[i][j] = y == 0 ? v : sum[i][j] + v;
            }
    }
    // only this block's registers of acc are looked at
    f32x4 acc[G::FI][G::FJ];
#pragma unroll
    for (int i = 0; i < G::FI; ++i)
#pragma unroll
        for (int j = 0; j < G::FJ; ++j) acc[i][j] = sum[i % 2][j];
    epi.template run<G>(acc, w, op, lds, lds + G::kStageBytes);
}

// ------------------------------------------------------------------------- plain epilogue -----
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b)
{
    const f16x2 v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float bf16_float(uint32_t bits) { return __uint_as_float(bits << 16); }

// A block of the wavefront's tile (32 rows) in FP32 in the LDS, 16-byte chunks
// XOR-permuted by the line: 16 lanes that write one chunk of 16 lines, or read every other chunk of two,
// meet 16 distinct bank groups.
template <class G>
struct Block32 {
    static constexpr int kRows = G::kBlockRows, kCols = G::kWaveCols;
    static constexpr int kLine = kCols * 4, kChunks = kLine / 16, kBytes = kRows * kLine;
    static constexpr int kBlocks = G::kWaveRows / kRows, BI = kRows / 16;
    // afterwards a lane takes eight columns of a line
    static constexpr int kLanes = kCols / 8, kLinesPerPass = 64 / kLanes, kPasses = kRows / kLinesPerPass;
    static_assert(kChunks == 16 || kChunks == 8, "the permutation below");
    static __device__ __forceinline__ int chunk(int line, int c)
    {
        return line * kLine + 16 * (c ^ (kChunks == 16 ? line & 15 : (line >> 1) & 7));
    }
    static __device__ __forceinline__ void get(const uint8_t *block, int line, int c8, f32x4 (&v)[2])
    {
        v[0] = *reinterpret_cast<const f32x4 *>(block + chunk(line, 2 * c8));
        v[1] = *reinterpret_cast<const f32x4 *>(block + chunk(line, 2 * c8 + 1));
    }
    // Block blk of the accumulators into the wavefront's part of the LDS. Registers have fixed names, so each
    // block has code of its own; the empty statements behind them differ, so that the compiler does not
    // make one piece of code with a variable index out of them (the accumulators would go to memory).
    static __device__ __forceinline__ void put(uint8_t *block, int lane, const f32x4 (&acc)[G::FI][G::FJ], int blk)
    {
        lds_order();   // what the lanes have read there before
        put_blocks(block + (lane & 15) * kLine, lane, acc, blk, std::make_integer_sequence<int, kBlocks>());
        lds_order();
    }

private:
    template <int... K>
    static __device__ __forceinline__ void put_blocks(uint8_t *line0, int lane, const f32x4 (&acc)[G::FI][G::FJ], int blk,
                                                      std::integer_sequence<int, K...>)
    {
        ((K == blk ? put_one<K>(line0, lane, acc, std::make_integer_sequence<int, BI * G::FJ>()) : void()), ...);
    }
    template <int K, int... E>
    static __device__ __forceinline__ void put_one(uint8_t *line0, int lane, const f32x4 (&acc)[G::FI][G::FJ],
                                                   std::integer_sequence<int, E...>)
    {
        const int r = lane & 15, q = lane >> 4;
        ((*reinterpret_cast<f32x4 *>(line0 + chunk(16 * (E / G::FJ) + r, 4 * (E % G::FJ) + q) - r * kLine) =
              acc[BI * K + E / G::FJ][E % G::FJ]),
         ...);
        asm volatile("; block %0" ::"i"(K));
    }
};

// c = alpha * A B^T + beta * c (+ add) in FP32 or bf16 (rounded once, after the sums); c is read only when
// beta != 0, add (FP32 [M][ld_add], 16-byte aligned rows, readable up to a multiple of 4 columns) only
// when it is not NULL. power: NULL, or an exponent in device memory: alpha 2^power takes the place of alpha.
template <bool BF16_OUT>
struct StoreEpi {
    static constexpr bool kSym = false;
    void *c;
    int64_t ldc, batch_c;   // elements
    float alpha, beta;
    const float *add = nullptr;
    int64_t ld_add = 0;
    const int *power = nullptr;

    template <class G>
    __device__ __forceinline__ void run(f32x4 (&acc)[G::FI][G::FJ], const Where &w, const Operands &op, uint8_t *lds,
                                        uint8_t *) const
    {
        run_with<G>(acc, w, op, lds, [](int, int) { return 0; }, [](f32x4 (&)[2], int) {});
    }

    // fetch(m, n): what make(v, fetched) wants to turn the product's eight values v at (m, n) into those that take
    // their place; m and n lie in the tile
    template <class G, class Fetch, class Make>
    __device__ __forceinline__ void run_with(f32x4 (&acc)[G::FI][G::FJ], const Where &w, const Operands &op, uint8_t *lds,
                                             Fetch fetch, Make make) const
    {
        using B = Block32<G>;
        uint8_t *block = lds + w.wave * G::kEpiWave;
        // an exponent of its own: 2^power may leave FP32's range where the result does not
        const int up = power ? *power : 0;
        const auto scaled = [&](f32x4 x) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = ldexpf(x[e] * alpha, up);
            return x;
        };
        constexpr int kElem = BF16_OUT ? 2 : 4;
        const bool vec = ldc % 8 == 0 && (uintptr_t)c % 16 == 0 && (batch_c % 8 == 0 || w.batch == 0);
        // the whole tile in 16-byte stores of nothing but the product
        const bool plain = vec && beta == 0.0f && !add && G::kTileM <= op.M - w.m0 && G::kTileN <= op.N - w.n0;
        const int line = w.lane / B::kLanes, c8 = w.lane % B::kLanes, n = w.n0 + w.col0 + 8 * c8;
#pragma unroll 1
        for (int blk = w.block0; blk < w.block1; ++blk) {
            // a block of the wavefront's rows through its part of the LDS (no barrier), so that a store
            // instruction writes whole lines; one code for all blocks: it is fetched for one use
            const int m = w.m0 + w.row0 + B::kRows * blk + line;
            if (plain) {
                decltype(fetch(0, 0)) got[B::kPasses];
#pragma unroll
                for (int p = 0; p < B::kPasses; ++p) got[p] = fetch(m + B::kLinesPerPass * p, n);
                B::put(block, w.lane, acc, blk);
                char *at = static_cast<char *>(c) + (w.batch * batch_c + (int64_t)m * ldc + n) * kElem;
#pragma unroll
                for (int p = 0; p < B::kPasses; ++p) {
                    f32x4 v[2];
                    B::get(block, B::kLinesPerPass * p + line, c8, v);
                    make(v, got[p]);
                    v[0] = scaled(v[0]);
                    v[1] = scaled(v[1]);
                    if constexpr (BF16_OUT) {
                        *reinterpret_cast<u32x4 *>(at) = u32x4{pack_bf16(v[0][0], v[0][1]), pack_bf16(v[0][2], v[0][3]),
                                                               pack_bf16(v[1][0], v[1][1]), pack_bf16(v[1][2], v[1][3])};
                    } else {
                        *reinterpret_cast<f32x4 *>(at) = v[0];
                        *reinterpret_cast<f32x4 *>(at + 16) = v[1];
                    }
                    at += B::kLinesPerPass * ldc * kElem;
                }
            } else {
                B::put(block, w.lane, acc, blk);
#pragma unroll 1
                for (int p = 0; p < B::kPasses; ++p) {
                    const int mm = m + B::kLinesPerPass * p;
                    if (mm >= op.M || n >= op.N) break;
                    f32x4 v[2];
                    B::get(block, B::kLinesPerPass * p + line, c8, v);
                    make(v, fetch(mm, n));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int nn = n + 4 * h;
                        if (nn >= op.N) break;
                        f32x4 x = scaled(v[h]);
                        if (add) x += *reinterpret_cast<const f32x4 *>(add + (int64_t)mm * ld_add + nn);
                        put(w.batch * batch_c + (int64_t)mm * ldc + nn, x, vec && nn + 4 <= op.N, op.N - nn);
                    }
                }
            }
        }
    }

    // four values at element `at`: at once (vec), or the first `count` of them one by one
    __device__ __forceinline__ void put(int64_t at, f32x4 v, bool vec, int count) const
    {
        if constexpr (BF16_OUT) {
            uint16_t *p = static_cast<uint16_t *>(c) + at;
            if (vec) {
                if (beta != 0.0f) {
                    const u32x2 old = *reinterpret_cast<const u32x2 *>(p);
                    v += beta * f32x4{bf16_float(old.x & 0xFFFFu), bf16_float(old.x >> 16), bf16_float(old.y & 0xFFFFu),
                                      bf16_float(old.y >> 16)};
                }
                *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                return;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < count) {
                    const float x = beta != 0.0f ? v[e] + beta * bf16_float(p[e]) : v[e];
                    p[e] = (uint16_t)(pack_bf16(x, 0.0f) & 0xFFFFu);
                }
        } else {
            float *p = static_cast<float *>(c) + at;
            if (vec) {
                if (beta != 0.0f) v += beta * *reinterpret_cast<const f32x4 *>(p);
                *reinterpret_cast<f32x4 *>(p) = v;
                return;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < count) p[e] = beta != 0.0f ? v[e] + beta * p[e] : v[e];
        }
    }
};

// ------------------------------------------------------------------- 16-bit tiles, two ways ---
// Writes the wavefront's part of the tile as 16-bit values, row-major at rows[m][ld_rows] and (cols !=
// nullptr) transposed at cols[n][ld_cols], m and n counted from the matrix' origin; every element of
// the tile has its place in both. fetch(m, n) reads what make(v, fetched, m, n) wants to turn the
// product's eight values v, columns n .. n + 7 of row m, into those to write; make may write
// row-major memory of its own there: the lanes of a row cover a line of 128 bytes. pack makes two
// values one word.
//
// A block of the accumulators goes through the LDS in FP32; one code serves all blocks, as it is fetched for
// one use. For the transposed a lane swaps four of its eight columns against the next row's, so that it holds
// two rows of four columns, and writes them as words where the block was; its lines are 64 bytes.
template <class G, class Pack, class Fetch, class Make>
__device__ __forceinline__ void store_tile16(f32x4 (&acc)[G::FI][G::FJ], const Where &w, uint8_t *lds, Pack pack, Fetch fetch,
                                             Make make, uint16_t *rows, int64_t ld_rows, uint16_t *cols, int64_t ld_cols)
{
    using B = Block32<G>;
    constexpr int kLine = B::kRows * 2, kPieces = kLine / 16;   // the transposed block: kCols lines
    uint8_t *block = lds + w.wave * G::kEpiWave;
    const int line = w.lane / B::kLanes, c8 = w.lane % B::kLanes, n = w.n0 + w.col0 + 8 * c8;
    const bool odd = line & 1;
    // 16-byte pieces of the transposed lines, XOR-permuted by the column
    const auto piece = [](int col, int p) { return col * kLine + 16 * (p ^ ((col >> 1) & (kPieces - 1))); };
    const auto next_row = [](uint32_t v) {
        if constexpr (B::kLanes == 8)
            return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x128, 0xF, 0xF, true);   // row_ror:8
        else
            return (uint32_t)__shfl_xor((int)v, B::kLanes);
    };
#pragma unroll 1
    for (int blk = w.block0; blk < w.block1; ++blk) {
        const int m = w.m0 + w.row0 + B::kRows * blk;
        decltype(fetch(0, 0)) got[B::kPasses];
#pragma unroll
        for (int p = 0; p < B::kPasses; ++p) got[p] = fetch(m + B::kLinesPerPass * p + line, n);
        B::put(block, w.lane, acc, blk);
        uint16_t *at = rows + (int64_t)(m + line) * ld_rows + n;
        uint32_t pairs[B::kPasses][4];
#pragma unroll
        for (int p = 0; p < B::kPasses; ++p) {
            const int l = B::kLinesPerPass * p + line;
            f32x4 v[2];
            B::get(block, l, c8, v);
            make(v, got[p], m + l, n);
            const uint32_t word[4] = {pack(v[0][0], v[0][1]), pack(v[0][2], v[0][3]), pack(v[1][0], v[1][1]),
                                      pack(v[1][2], v[1][3])};
            *reinterpret_cast<u32x4 *>(at) = u32x4{word[0], word[1], word[2], word[3]};
            at += B::kLinesPerPass * ld_rows;
            if (cols) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // even lines keep columns 0 .. 3 and get those of the line below; odd ones keep 4 .. 7
                    const uint32_t got_word = next_row(odd ? word[h] : word[2 + h]);
                    const uint32_t up = odd ? got_word : word[h], dn = odd ? word[2 + h] : got_word;
                    pairs[p][2 * h] = __builtin_amdgcn_perm(dn, up, 0x05040100u);
                    pairs[p][2 * h + 1] = __builtin_amdgcn_perm(dn, up, 0x07060302u);
                }
            }
        }
        if (cols) {
            lds_order();
#pragma unroll
            for (int p = 0; p < B::kPasses; ++p)
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int c = 8 * c8 + (odd ? 4 : 0) + h, l = (B::kLinesPerPass * p + line) & ~1;
                    *reinterpret_cast<uint32_t *>(block + piece(c, l >> 3) + 2 * (l & 7)) = pairs[p][h];
                }
            lds_order();
            constexpr int kColsPerPass = 64 / kPieces;
            const int col = w.lane / kPieces, pc = w.lane % kPieces;
            uint16_t *to = cols + (int64_t)(w.n0 + w.col0 + col) * ld_cols + m + 8 * pc;
#pragma unroll
            for (int p = 0; p < B::kCols / kColsPerPass; ++p)
                *reinterpret_cast<u32x4 *>(to + (int64_t)kColsPerPass * p * ld_cols) =
                    *reinterpret_cast<const u32x4 *>(block + piece(kColsPerPass * p + col, pc));
        }
    }
}

// ---------------------------------------------------------------------------------- launch ----
// What runs a product: the tile, how many tiles have a workgroup each, and how many workgroups share each of
// the others.
struct Plan {
    int geo;      // 0 Big, 1 Small, 2 Tiny
    int whole, tail, splits, per;
    size_t partial_bytes;
};
constexpr int kTileSide[3] = {256, 128, 64};
constexpr int kThreads[3] = {64 * Big::NW, 64 * Small::NW, 64 * Tiny::NW};

inline int64_t count_tiles(int64_t M, int64_t N, bool sym, int side)
{
    const int64_t tm = (M + side - 1) / side, tn = (N + side - 1) / side;
    return sym ? tm * (tm + 1) / 2 : tm * tn;
}

// A round of n workgroups of one tile size, `per` stages each, in microseconds: so much for a stage and so
// much around the stages, with how many workgroups share a CU. Measured in bf16: 16 workgroups of 256 x 256
// take 1.02 a stage, 256 of them 1.45 by the power cap, and 136 of them 1.44 in a run of such products,
// which the cap holds down for longer than one of them lasts; 128 x 128: 16 take 0.44, 256 0.50, 512 0.95 to
// 1.05, 416 over a contraction of 50304 1.34; 64 x 64: 0.18, 0.20 and 0.36.
inline double round_time(int geo, int64_t n, int64_t per)
{
    const double share = (double)n / kComputeUnits;
    switch (geo) {
    case 0: return (double)per * (1.02 + 0.43 * (share < 0.5 ? 2.0 * share : 1.0)) + 8.0 + 3.0 * share;
    case 1: return (double)per * (share > 1.0 ? 0.50 + 0.70 * (share - 1.0) : 0.50) + 4.5 + 2.0 * share;
    default: return (double)per * (share > 1.0 ? 0.20 + 0.16 * (share - 1.0) : 0.20) + 4.0 + 0.8 * share;
    }
}

// The plan with the least time by that account (whole < 0: the product has more tiles than a grid): full rounds of as many workgroups as the chip holds, and the
// tiles left over, each worked by several workgroups if that is quicker; then their sums' kernel too, whose
// workgroups read one split after the other (0.9, 0.5 and 0.3 us each by tile size). 1024 x 1024 x
// 8192: 137 us in 256 x 256 tiles, 54 split eight ways, 35 in 128 x 128 tiles split four ways, 30 in 64 x 64
// unsplit; 1537 x 1024 x 50304: 811, 195 split nine ways, 216 in 128 x 128 split four ways.
inline Plan plan_product(int64_t M, int64_t N, int64_t nk, bool sym, int64_t batch)
{
    constexpr int kSlots[3] = {kComputeUnits, 2 * kComputeUnits, 2 * kComputeUnits};
    constexpr double kJoin[3] = {0.9, 0.5, 0.3};
    Plan best{0, -1, 0, 1, 1, 0};
    double least = 0.0;
    if (nk < 1) nk = 1;   // an empty contraction asks for no workspace
    // more tiles than a grid has in any of the sizes: no plan
    if ((double)M * (double)N * (double)batch > 1e15) return Plan{0, -1, 0, 1, (int)nk, 0};
    for (int g = 0; g < 3; ++g) {
        const int64_t tiles = count_tiles(M, N, sym, kTileSide[g]) * batch;
        if (tiles > kMaxItems / kThreads[g]) continue;
        const int64_t full = tiles / kSlots[g] * kSlots[g], left = tiles - full;
        const double rounds = (double)(tiles / kSlots[g]) * round_time(g, kSlots[g], nk);
        double t = rounds + (left ? round_time(g, left, nk) : 0.0);
        if (least == 0.0 || t < least) {
            least = t;
            best = Plan{g, (int)tiles, 0, 1, (int)nk, 0};
        }
        for (int64_t s = 2; s <= 16 && left > 0 && nk / s >= 4; ++s) {
            const int64_t per = (nk + s - 1) / s, used = (nk + per - 1) / per, n = left * used;
            if (used != s || full + n > kMaxItems / kThreads[g]) continue;
            const double bytes = (double)n * kTileSide[g] * kTileSide[g] * 4;
            t = rounds + (double)(n / kSlots[g]) * round_time(g, kSlots[g], per) +
                (n % kSlots[g] ? round_time(g, n % kSlots[g], per) : 0.0) + 3.0 + (double)used * kJoin[g] + bytes / 4.0e6;
            if (t < least) {
                least = t;
                best = Plan{g, (int)full, (int)left, (int)used, (int)per, (size_t)bytes};
            }
        }
    }
    return best;
}
// The same tile without the workspace.
inline Plan unsplit(Plan p, int64_t nk)
{
    return Plan{p.geo, p.whole + p.tail, 0, 1, (int)nk, 0};
}

template <class E, class G, class Epi>
hipError_t launch_planned(Operands op, const Epi &epi, const Plan &plan, void *partials, hipStream_t stream)
{
    op.tiles_m = (op.M - 1) / G::kTileM + 1;   // M + 255 may leave 32 bits
    op.tiles_n = (op.N - 1) / G::kTileN + 1;
    if (plan.whole < 0) return hipErrorInvalidValue;
    op.whole = plan.whole;
    op.splits = plan.splits;
    op.per = plan.per;
    op.partials = static_cast<f32x4 *>(partials);
    const unsigned grid = (unsigned)plan.whole + (unsigned)plan.tail * (unsigned)plan.splits;
    const hipError_t e = launch(product_kernel<E, G, Epi>, dim3(grid), dim3(64 * G::NW), 0, stream, op, epi);
    if (e != hipSuccess || plan.tail == 0) return e;
    return launch(finish_kernel<G, Epi>, dim3((unsigned)(plan.tail * G::kEpiBlocks)), dim3(64 * G::NW), 0, stream, op, epi);
}

// partials: room for plan.partial_bytes (NULL when the plan does not split)
template <class E, class Epi>
hipError_t launch_product(const Operands &op, const Epi &epi, const Plan &plan, void *partials, hipStream_t stream)
{
    switch (plan.geo) {
    case 0: return launch_planned<E, Big>(op, epi, plan, partials, stream);
    case 1: return launch_planned<E, Small>(op, epi, plan, partials, stream);
    default: return launch_planned<E, Tiny>(op, epi, plan, partials, stream);
    }
}

}  // namespace slab
}  // namespace mx
