// The norm over many gradients together, and the gradients scaled down to a largest norm.
//
//   n = sqrt(sum over all values of g^2),  c = min(1, max_norm / (n + eps)),  out = c g
//
// Squares are summed in 64 bits: the square of an FP32 value is exact there, and cannot overflow. The sums do not
// depend on the run: every workgroup adds its own share of the values, and the workgroups' sums are added in a fixed order.
#include <algorithm>
#include <cstdint>
#include <vector>

#include "internal.h"
#include "layer_device.h"

namespace mx {
namespace {

// A launch has at most two workgroups a CU, and all of them are at neighbouring pieces at any time: 872 MB of FP32 values into bf16
// ones take 355 to 365 us (with eight workgroups a CU, each at a run of pieces of its own, 423; with one 352, but then 105 million bf16
// values 126 instead of 101). The scaling goes from the last piece to the first: it begins with what the sums have left in the last
// cache, and what it writes does not stay there if that is too much (372 us; 397 without such stores).
constexpr int64_t kPiece = 8192;                // values that a workgroup of 256 threads works at a time
constexpr int64_t kMostBlocks = 512;            // workgroups of a launch, and so partial sums

// A launch's tensors, in a kernel's 4 KB of arguments: 16 bytes each for the sums, 24 with an output (300 tensors in four launches
// take 22 us on the GPU, 162 with the host's part; with 28 bytes each, in six, 28 and 170).
template <int N, bool OUT>
struct Tensors {
    static constexpr int kMost = N;
    const void *g[N];
    void *out[OUT ? N : 1];
    uint32_t first[N + 1];                      // pieces before each
    uint32_t f32[N / 32], out_f32[N / 32];
    uint32_t last[N];                           // values of the last piece
    int n;
    // values of piece i, which is tensor k's
    __device__ __forceinline__ int count(uint32_t i, int k) const { return i + 1 == first[k + 1] ? (int)last[k] : (int)kPiece; }
};
typedef Tensors<224, false> Inputs;
typedef Tensors<160, true> Pairs;
static_assert(sizeof(Inputs) <= 4000 && sizeof(Pairs) <= 4000, "a kernel's arguments");

// the tensor that holds piece `i`: as many as end before it, counted by the lanes at once
template <class T>
__device__ __forceinline__ int tensor_of(const T &t, uint32_t i)
{
    int k = 0;
    for (int j = 0; j < t.n - 1; j += 64) {
        const int lane = j + ((int)threadIdx.x & 63);
        k += __popcll(__ballot(lane < t.n - 1 && t.first[lane + 1] <= i));
    }
    return __builtin_amdgcn_readfirstlane(k);
}

__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double part[4];
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

template <bool F32>
__device__ __forceinline__ double piece_squares(const void *g, int count)
{
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < (int)(kPiece / 2048); ++k) {
        float v[8];
        load_raw<F32, true>(g, k * 2048 + 8 * (int)threadIdx.x, count).get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fma((double)v[e], (double)v[e], sum);
    }
    return sum;
}

__global__ __launch_bounds__(256) void squares_kernel(Inputs t, double *part)
{
    const uint32_t end = t.first[t.n];
    double sum = 0.0;
    for (uint32_t i = blockIdx.x, k = tensor_of(t, i); i < end; i += gridDim.x) {
        while (t.first[k + 1] <= i) ++k;
        const int64_t at0 = (int64_t)(i - t.first[k]) * kPiece;
        sum += (t.f32[k / 32] >> (k % 32)) & 1 ? piece_squares<true>(at<true>(t.g[k], at0), t.count(i, k))
                                               : piece_squares<false>(at<false>(t.g[k], at0), t.count(i, k));
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// the sum of `count` partial sums, by every workgroup that needs it: always in the same order
__device__ __forceinline__ double join(const double *part, int count)
{
    double sum = 0.0;
    for (int i = threadIdx.x; i < count; i += 256) sum += part[i];
    return block_sum(sum);
}

__global__ __launch_bounds__(256) void join_kernel(const double *part, int count, double *sum_sq, float *norm)
{
    const double sum = join(part, count);
    if (threadIdx.x) return;
    if (sum_sq) *sum_sq = sum;
    if (norm) *norm = (float)sqrt(sum);
}

// values times c 2^e2
template <bool F32, bool OUT, bool NT>
__device__ __forceinline__ void scale_piece(const void *g, void *out, int64_t at0, int count, float c, int e2)
{
    g = at<F32>(g, at0);
    out = at<OUT>(out, at0);
    Raw8<F32> r[kPiece / 2048];
#pragma unroll
    for (int k = 0; k < (int)(kPiece / 2048); ++k)
        r[k] = load_raw<F32, true>(g, k * 2048 + 8 * (int)threadIdx.x, count);
#pragma unroll
    for (int k = 0; k < (int)(kPiece / 2048); ++k) {
        float v[8];
        r[k].get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= c;
        if (e2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = ldexpf(v[e], e2);
        }
        Raw8<OUT> o;
        o.set(v);
        store_raw<OUT, true, NT>(o, out, k * 2048 + 8 * (int)threadIdx.x, count);
    }
}

template <bool NT>
__global__ __launch_bounds__(256) void scale_kernel(Pairs t, const double *part, int parts, double max_norm, double eps,
                                                    float *norm)
{
    const double n = sqrt(join(part, parts));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
    // a norm that is NaN makes everything NaN
    const double q = max_norm / (n + eps);
    // a factor below FP32's normal range would lose bits that the products have: its exponent is applied to them (for all lanes
    // or none, so that other factors pay nothing)
    int e2 = 0;
    const float c = q > 1.0 ? 1.0f : (float)(q < 0x1p-126 ? frexp(q, &e2) : q);
    e2 = __builtin_amdgcn_readfirstlane(e2);
    const int end = (int)t.first[t.n];
    int i = end - 1 - (int)blockIdx.x;
    for (int k = tensor_of(t, (uint32_t)max(i, 0)); i >= 0; i -= (int)gridDim.x) {
        while (t.first[k] > (uint32_t)i) --k;
        if (c == 1.0f && e2 == 0 && t.g[k] == t.out[k]) continue;      // in place and nothing to do
        const int64_t at0 = (int64_t)((uint32_t)i - t.first[k]) * kPiece;
        const int count = t.count((uint32_t)i, k);
        const bool f32 = (t.f32[k / 32] >> (k % 32)) & 1, o32 = (t.out_f32[k / 32] >> (k % 32)) & 1;
        if (f32)
            o32 ? scale_piece<true, true, NT>(t.g[k], t.out[k], at0, count, c, e2)
                : scale_piece<true, false, NT>(t.g[k], t.out[k], at0, count, c, e2);
        else
            o32 ? scale_piece<false, true, NT>(t.g[k], t.out[k], at0, count, c, e2)
                : scale_piece<false, false, NT>(t.g[k], t.out[k], at0, count, c, e2);
    }
}

int64_t pieces(int64_t count) { return (count + kPiece - 1) / kPiece; }

// The end of the launch that begins with item i: as many as it holds, and fewer than 2^31 pieces, of which each has at most 2^24.
int64_t launch_end(const GradItem *items, int64_t n, int64_t i, int most)
{
    const int64_t end = std::min(n, i + most);
    for (int64_t total = 0; i < end; ++i)
        if ((total += pieces(items[i].count)) > INT32_MAX) break;
    return i;
}

// Sets t to these items and returns the launch's workgroups.
template <class T>
unsigned set_launch(const GradItem *items, int64_t n, T &t)
{
    t = T{};
    int64_t total = 0;
    for (; t.n < n; t.first[++t.n] = (uint32_t)total) {
        const GradItem &item = items[t.n];
        const int64_t p = pieces(item.count);
        t.g[t.n] = item.g;
        t.f32[t.n / 32] |= (uint32_t)item.f32 << (t.n % 32);
        if (sizeof(t.out) > sizeof(void *)) {
            t.out[t.n] = item.out;
            t.out_f32[t.n / 32] |= (uint32_t)item.out_f32 << (t.n % 32);
        }
        t.last[t.n] = (uint32_t)(item.count - (p - 1) * kPiece);
        total += p;
    }
    return (unsigned)std::min(total, kMostBlocks);
}

hipError_t launch_squares(const GradItem *items, int64_t n, double *part, int &count, hipStream_t stream)
{
    Inputs t;
    count = 0;
    for (int64_t i = 0, end; i < n; i = end) {
        end = launch_end(items, n, i, Inputs::kMost);
        const unsigned blocks = set_launch(items + i, end - i, t);
        if (hipError_t e = launch(squares_kernel, dim3(blocks), dim3(256), 0, stream, t, part + count)) return e;
        count += (int)blocks;
    }
    return hipSuccess;
}

hipError_t launch_scale(const GradItem *items, int64_t n, const double *part, int count, float max_norm, float eps,
                        float *norm, hipStream_t stream)
{
    int64_t bytes = 0;
    for (int64_t i = 0; i < n; ++i) bytes += items[i].count * ((items[i].f32 ? 4 : 2) + (items[i].out_f32 ? 4 : 2));
    const auto kernel = bytes > kStreamBytes ? scale_kernel<true> : scale_kernel<false>;
    // the launches too go from the last tensors to the first
    std::vector<int64_t> ends{0};
    while (ends.back() < n) ends.push_back(launch_end(items, n, ends.back(), Pairs::kMost));
    if (n == 0) ends.push_back(0);               // one writes the norm
    Pairs t;
    for (size_t k = ends.size() - 1; k > 0; --k) {
        const unsigned blocks = std::max(set_launch(items + ends[k - 1], ends[k] - ends[k - 1], t), 1u);
        if (hipError_t e = launch(kernel, dim3(blocks), dim3(256), 0, stream, t, part, count, (double)max_norm, (double)eps, norm))
            return e;
        norm = nullptr;
    }
    return hipSuccess;
}

}  // namespace

size_t grad_norm_workspace_bytes(const GradItem *items, int64_t n)
{
    int64_t blocks = 0;
    for (int64_t i = 0, end; i < n; i = end) {
        end = launch_end(items, n, i, Inputs::kMost);
        int64_t total = 0;
        for (int64_t k = i; k < end; ++k) total += pieces(items[k].count);
        blocks += std::min(total, kMostBlocks);
    }
    return (size_t)(blocks + 1) * sizeof(double);
}

hipError_t launch_grad_norm(const GradItem *items, int64_t n, void *ws, double *sum_sq, float *norm, hipStream_t stream)
{
    double *part = static_cast<double *>(ws);
    int count;
    if (hipError_t e = launch_squares(items, n, part, count, stream)) return e;
    return launch(join_kernel, dim3(1), dim3(256), 0, stream, static_cast<const double *>(part), count, sum_sq, norm);
}

hipError_t launch_grad_scale(const GradItem *items, int64_t n, const double *sum_sq, float max_norm, float eps, float *norm,
                             hipStream_t stream)
{
    return launch_scale(items, n, sum_sq, 1, max_norm, eps, norm, stream);
}

hipError_t launch_grad_clip(const GradItem *items, int64_t n, float max_norm, float eps, void *ws, float *norm, hipStream_t stream)
{
    double *part = static_cast<double *>(ws);
    int count;
    if (hipError_t e = launch_squares(items, n, part, count, stream)) return e;
    // every workgroup joins few sums by itself; many are joined once, into the place behind them
    if (count > 4096) {
        if (hipError_t e = launch(join_kernel, dim3(1), dim3(256), 0, stream, static_cast<const double *>(part), count, part + count, (float *)nullptr))
            return e;
        return launch_scale(items, n, part + count, 1, max_norm, eps, norm, stream);
    }
    return launch_scale(items, n, part, count, max_norm, eps, norm, stream);
}

}  // namespace mx
