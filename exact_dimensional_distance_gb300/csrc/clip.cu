// Clipping by the global gradient norm over many tensors.
#include <algorithm>

#include "hiss_internal.cuh"
#include "numeric.cuh"

namespace hiss {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 64;  // per tensor

// Partial sums of squares of one tensor, one per block, in float64.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_sum_squares(const T *x, int64_t n, double *part)
{
    __shared__ double warp_sum[kThreads / 32];
    double s = 0.0;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const double v = to_f32(x[i]);
        s += v * v;
    }
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) s += warp_sum[w];
        part[blockIdx.x] = s;
    }
}

// The norm from the partial sums, and the factor of every gradient.
__global__ void __launch_bounds__(kThreads) k_clip_factor(const double *part, int64_t n, float max_norm, float *norm,
                                                          float *factor)
{
    __shared__ double sum[kThreads];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) s += part[i];
    sum[threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kThreads; ++i) s += sum[i];
        const double v = sqrt(s);
        *norm = (float)v;
        *factor = isfinite(v) && v > (double)max_norm ? (float)((double)max_norm / v) : 1.0f;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_scale(const T *x, T *y, int64_t n, const float *factor)
{
    const float f = *factor;
    if (f == 1.0f && x == y) return;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads)
        y[i] = f == 1.0f ? x[i] : from_f32<T>(to_f32(x[i]) * f);
}

}  // namespace

size_t clip_tmp_bytes(const hiss_tensor *, int64_t count) { return 8 * (size_t)(count * kBlocks) + 16; }

cudaError_t clip_grads(const hiss_tensor *t, int64_t count, float max_norm, float *norm, void *tmp, cudaStream_t s,
                       int64_t *launches)
{
    double *part = static_cast<double *>(tmp) + 2;
    float *factor = static_cast<float *>(tmp);
    int64_t used = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (t[i].n == 0) continue;
        HISS_TRY(with_dtype(t[i].dtype, [&](auto e) {
            using T = decltype(e);
            k_sum_squares<T><<<kBlocks, kThreads, 0, s>>>(static_cast<const T *>(t[i].in), t[i].n, part + used * kBlocks);
            return cudaGetLastError();
        }));
        ++used;
    }
    k_clip_factor<<<1, kThreads, 0, s>>>(part, used * kBlocks, max_norm, norm, factor);
    *launches += used + 1;
    for (int64_t i = 0; i < count; ++i) {
        if (t[i].n == 0) continue;
        HISS_TRY(with_dtype(t[i].dtype, [&](auto e) {
            using T = decltype(e);
            const T *in = static_cast<const T *>(t[i].in);
            T *out = t[i].out ? static_cast<T *>(t[i].out) : const_cast<T *>(in);
            k_scale<T><<<(unsigned)std::min<int64_t>(152 * 8, (t[i].n + kThreads - 1) / kThreads), kThreads, 0, s>>>(
                in, out, t[i].n, factor);
            return cudaGetLastError();
        }));
        ++*launches;
    }
    return cudaGetLastError();
}

}  // namespace hiss
