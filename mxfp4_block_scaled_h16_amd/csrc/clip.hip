// The norm over many gradients together, and the gradients scaled down to a largest norm.
//
//   n = sqrt(sum over all values of g^2),  c = min(1, max_norm / (n + eps)),  out = c g
//
// Squares are summed in 64 bits: the square of an FP32 value is exact there, and cannot overflow. The sums do not
// depend on the run: every workgroup adds its own share of the values, and the workgroups' sums are added in a fixed order.
#include <algorithm>

#include "internal.h"
#include "layer_device.h"

namespace mx {
namespace {

constexpr int kTensors = 128;                   // a launch's tensors (28 bytes each of a kernel's 4 KB of arguments)
constexpr int64_t kPiece = 8192;                // values that a workgroup of 256 threads works at a time
constexpr int64_t kMostBlocks = 2048;           // workgroups of a launch, and so partial sums

struct Tensors {
    const void *g[kTensors];
    void *out[kTensors];
    int64_t count[kTensors];
    uint32_t first[kTensors + 1];               // pieces before each
    uint32_t f32[kTensors / 32], out_f32[kTensors / 32];
    int n;
    uint32_t per_block;                         // pieces of a workgroup, side by side
};
static_assert(sizeof(Tensors) <= 4000, "a kernel's arguments");

// the tensor that holds piece `i`
__device__ __forceinline__ int tensor_of(const Tensors &t, uint32_t i)
{
    int lo = 0, hi = t.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.first[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
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
    uint32_t i = blockIdx.x * t.per_block;
    const uint32_t end = min(i + t.per_block, t.first[t.n]);
    double sum = 0.0;
    for (int k = i < end ? tensor_of(t, i) : 0; i < end; ++i) {
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

template <bool F32, bool OUT>
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
        store_raw<OUT, true>(o, out, at0 + k * 2048 + 8 * (int)threadIdx.x, count);
    }
}

__global__ __launch_bounds__(256) void scale_kernel(Tensors t, const double *part, int count, double max_norm, double eps,
                                                    float *norm)
{
    const double n = sqrt(join(part, count));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
    // a norm that is NaN makes everything NaN
    const double q = max_norm / (n + eps);
    const float c = q > 1.0 ? 1.0f : (float)q;
    uint32_t i = blockIdx.x * t.per_block;
    const uint32_t end = min(i + t.per_block, t.first[t.n]);
    for (int k = i < end ? tensor_of(t, i) : 0; i < end; ++i) {
        while (t.first[k + 1] <= i) ++k;
        if (c == 1.0f && t.g[k] == t.out[k]) continue;      // in place and nothing to do
        const int64_t at0 = (int64_t)(i - t.first[k]) * kPiece;
        const bool f32 = (t.f32[k / 32] >> (k % 32)) & 1, o32 = (t.out_f32[k / 32] >> (k % 32)) & 1;
        if (f32)
            o32 ? scale_piece<true, true>(t.g[k], t.out[k], at0, t.count[k], c)
                : scale_piece<true, false>(t.g[k], t.out[k], at0, t.count[k], c);
        else
            o32 ? scale_piece<false, true>(t.g[k], t.out[k], at0, t.count[k], c)
                : scale_piece<false, false>(t.g[k], t.out[k], at0, t.count[k], c);
    }
}

int64_t pieces(int64_t count) { return (count + kPiece - 1) / kPiece; }

// The next launch's tensors, from item i on: as many as one holds, fewer than 2^31 pieces. Returns its workgroups.
unsigned next_launch(const GradItem *items, int64_t n, int64_t &i, Tensors &t)
{
    t = Tensors{};
    int64_t total = 0;
    for (; i < n && t.n < kTensors; ++i) {
        t.g[t.n] = items[i].g;
        t.out[t.n] = items[i].out;
        t.count[t.n] = items[i].count;
        t.f32[t.n / 32] |= (uint32_t)items[i].f32 << (t.n % 32);
        t.out_f32[t.n / 32] |= (uint32_t)items[i].out_f32 << (t.n % 32);
        total += pieces(items[i].count);
        t.first[++t.n] = (uint32_t)total;
    }
    t.per_block = (uint32_t)((total + kMostBlocks - 1) / kMostBlocks);
    return t.per_block ? (unsigned)((total + t.per_block - 1) / t.per_block) : 0u;
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
    Tensors t;
    int64_t i = 0;
    do {
        const unsigned blocks = std::max(next_launch(items, n, i, t), 1u);   // one writes the norm
        if (hipError_t e = launch(scale_kernel, dim3(blocks), dim3(256), 0, stream, t, part, count, (double)max_norm, (double)eps, norm))
            return e;
        norm = nullptr;
    } while (i < n);
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
    if (count > (int)(2 * kMostBlocks)) {
        if (hipError_t e = launch(join_kernel, dim3(1), dim3(256), 0, stream, static_cast<const double *>(part), count, part + count, (float *)nullptr))
            return e;
        return launch_scale(items, n, part + count, 1, max_norm, eps, norm, stream);
    }
    return launch_scale(items, n, part, count, max_norm, eps, norm, stream);
}

}  // namespace mx
