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
// ones take 355 us (with eight workgroups a CU, each at a run of pieces of its own, 423; with one 352, but then 105 million bf16
// values 126 instead of 101). The scaling goes from the last piece to the first: it begins with what the sums have left in the last
// cache, and what it writes does not stay there if that is too much (372 us; 397 without such stores).
constexpr int kTensors = 128;                   // a launch's tensors (28 bytes each of a kernel's 4 KB of arguments)
constexpr int64_t kPiece = 8192;                // values that a workgroup of 256 threads works at a time
constexpr int64_t kMostBlocks = 512;            // workgroups of a launch, and so partial sums

struct Tensors {
    const void *g[kTensors];
    void *out[kTensors];
    int64_t count[kTensors];
    uint32_t first[kTensors + 1];               // pieces before each
    uint32_t f32[kTensors / 32], out_f32[kTensors / 32];
    int n;
};
static_assert(sizeof(Tensors) <= 4000, "a kernel's arguments");

// the tensor that holds piece `i`: as many as end before it, counted by the lanes at once
__device__ __forceinline__ int tensor_of(const Tensors &t, uint32_t i)
{
    int k = 0;
#pragma unroll
    for (int j = 0; j < kTensors; j += 64) {
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
__device__ __forceinline__ double piece_squares(const void *g, int64_t at0, int64_t count)
{
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < (int)(kPiece / 2048); ++k) {
        float v[8];
        load_raw<F32, true>(g, at0 + k * 2048 + 8 * (int)threadIdx.x, count).get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fma((double)v[e], (double)v[e], sum);
    }
    return sum;
}

__global__ __launch_bounds__(256) void squares_kernel(Tensors t, double *part)
{
    const uint32_t end = t.first[t.n];
    double sum = 0.0;
    for (uint32_t i = blockIdx.x, k = tensor_of(t, i); i < end; i += gridDim.x) {
        while (t.first[k + 1] <= i) ++k;
        const int64_t at0 = (int64_t)(i - t.first[k]) * kPiece;
        sum += (t.f32[k / 32] >> (k % 32)) & 1 ? piece_squares<true>(t.g[k], at0, t.count[k])
                                               : piece_squares<false>(t.g[k], at0, t.count[k]);
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

template <bool F32, bool OUT, bool NT>
__device__ __forceinline__ void scale_piece(const void *g, void *out, int64_t at0, int64_t count, float c)
{
    Raw8<F32> r[kPiece / 2048];
#pragma unroll
    for (int k = 0; k < (int)(kPiece / 2048); ++k)
        r[k] = load_raw<F32, true>(g, at0 + k * 2048 + 8 * (int)threadIdx.x, count);
#pragma unroll
    for (int k = 0; k < (int)(kPiece / 2048); ++k) {
        float v[8];
        r[k].get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= c;
        Raw8<OUT> o;
        o.set(v);
        store_raw<OUT, true, NT>(o, out, at0 + k * 2048 + 8 * (int)threadIdx.x, count);
    }
}

template <bool NT>
__global__ __launch_bounds__(256) void scale_kernel(Tensors t, const double *part, int count, double max_norm, double eps,
                                                    float *norm)
{
    const double n = sqrt(join(part, count));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
    // a norm that is NaN makes everything NaN
    const double q = max_norm / (n + eps);
    const float c = q > 1.0 ? 1.0f : (float)q;
    const int end = (int)t.first[t.n];
    int i = end - 1 - (int)blockIdx.x;
    for (int k = tensor_of(t, (uint32_t)max(i, 0)); i >= 0; i -= (int)gridDim.x) {
        while (t.first[k] > (uint32_t)i) --k;
        if (c == 1.0f && t.g[k] == t.out[k]) continue;      // in place and nothing to do
        const int64_t at0 = (int64_t)((uint32_t)i - t.first[k]) * kPiece;
        const bool f32 = (t.f32[k / 32] >> (k % 32)) & 1, o32 = (t.out_f32[k / 32] >> (k % 32)) & 1;
        if (f32)
            o32 ? scale_piece<true, true, NT>(t.g[k], t.out[k], at0, t.count[k], c)
                : scale_piece<true, false, NT>(t.g[k], t.out[k], at0, t.count[k], c);
        else
            o32 ? scale_piece<false, true, NT>(t.g[k], t.out[k], at0, t.count[k], c)
                : scale_piece<false, false, NT>(t.g[k], t.out[k], at0, t.count[k], c);
    }
}

int64_t pieces(int64_t count) { return (count + kPiece - 1) / kPiece; }

// The launch of the tensors from item i on, as many as one holds (fewer than 2^31 pieces, each having at most 2^24): sets i behind
// them and returns its workgroups.
unsigned next_launch(const GradItem *items, int64_t n, int64_t &i, Tensors &t)
{
    t = Tensors{};
    int64_t total = 0;
    for (; i < n && t.n < kTensors; ++i) {
        if (total + pieces(items[i].count) > INT32_MAX) break;
        t.g[t.n] = items[i].g;
        t.out[t.n] = items[i].out;
        t.count[t.n] = items[i].count;
        t.f32[t.n / 32] |= (uint32_t)items[i].f32 << (t.n % 32);
        t.out_f32[t.n / 32] |= (uint32_t)items[i].out_f32 << (t.n % 32);
        total += pieces(items[i].count);
        t.first[++t.n] = (uint32_t)total;
    }
    return (unsigned)std::min(total, kMostBlocks);
}

hipError_t launch_squares(const GradItem *items, int64_t n, double *part, int &count, hipStream_t stream)
{
    Tensors t;
    count = 0;
    for (int64_t i = 0; i < n;) {
        const unsigned blocks = next_launch(items, n, i, t);
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
    std::vector<int64_t> starts;
    Tensors t;
    for (int64_t i = 0; i < n;) {
        starts.push_back(i);
        next_launch(items, n, i, t);
    }
    if (starts.empty()) starts.push_back(0);     // one writes the norm
    for (size_t k = starts.size(); k-- > 0;) {
        int64_t i = starts[k];
        const unsigned blocks = std::max(next_launch(items, n, i, t), 1u);
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
    Tensors t;
    for (int64_t i = 0; i < n;) blocks += next_launch(items, n, i, t);
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
