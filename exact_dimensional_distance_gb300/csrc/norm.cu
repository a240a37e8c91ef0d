// Layer norm, forward and backward.
#include "hiss_internal.cuh"
#include "numeric.cuh"

namespace hiss {
namespace {

constexpr int kThreads = 256;

// Sum of v over the block, returned to every thread.
__device__ __forceinline__ float block_sum(float v)
{
    __shared__ float part[kThreads / 32];
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < kThreads / 32; ++w) s += part[w];
    return s;
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(kThreads) k_norm(NormArgs a)
{
    const int64_t r = blockIdx.x;
    const TX *x = static_cast<const TX *>(a.x) + r * a.x_stride;
    float s = 0.0f;
    for (int c = threadIdx.x; c < a.width; c += kThreads) s += to_f32(x[c]);
    const float mean = block_sum(s) / a.width;
    s = 0.0f;
    for (int c = threadIdx.x; c < a.width; c += kThreads) {
        const float e = to_f32(x[c]) - mean;
        s += e * e;
    }
    const float rstd = 1.0f / sqrtf(block_sum(s) / a.width + a.eps);
    TY *y = static_cast<TY *>(a.y) + r * a.y_stride;
    for (int c = threadIdx.x; c < a.width; c += kThreads) {
        float v = (to_f32(x[c]) - mean) * rstd;
        if (a.weight) v *= load_any(a.weight, a.p_dtype, c);
        if (a.bias) v += load_any(a.bias, a.p_dtype, c);
        y[c] = from_f32<TY>(v);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
    }
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(kThreads) k_norm_dx(NormArgs a)
{
    const int64_t r = blockIdx.x;
    const TX *x = static_cast<const TX *>(a.x) + r * a.x_stride;
    const TY *dy = static_cast<const TY *>(a.dy) + r * a.y_stride;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float sg = 0.0f, sgh = 0.0f;
    for (int c = threadIdx.x; c < a.width; c += kThreads) {
        const float g = to_f32(dy[c]) * (a.weight ? load_any(a.weight, a.p_dtype, c) : 1.0f);
        sg += g;
        sgh += g * ((to_f32(x[c]) - mean) * rstd);
    }
    const float mg = block_sum(sg) / a.width, mgh = block_sum(sgh) / a.width;
    TX *dx = static_cast<TX *>(a.dx) + r * a.dx_stride;
    for (int c = threadIdx.x; c < a.width; c += kThreads) {
        const float g = to_f32(dy[c]) * (a.weight ? load_any(a.weight, a.p_dtype, c) : 1.0f);
        dx[c] = from_f32<TX>(rstd * (g - mg - (to_f32(x[c]) - mean) * rstd * mgh));
    }
}

// 32 columns per block, 8 rows at a time.
template <typename TX, typename TY>
__global__ void __launch_bounds__(kThreads) k_norm_dparam(NormArgs a)
{
    __shared__ float sw[8][33], sb[8][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float dw = 0.0f, db = 0.0f;
    if (c < a.width)
        for (int64_t r = w; r < a.n; r += 8) {
            const float dy = to_f32(static_cast<const TY *>(a.dy)[r * a.y_stride + c]);
            db += dy;
            dw += dy * ((to_f32(static_cast<const TX *>(a.x)[r * a.x_stride + c]) - a.mean[r]) * a.rstd[r]);
        }
    sw[w][lane] = dw;
    sb[w][lane] = db;
    __syncthreads();
    if (w == 0 && c < a.width) {
        for (int i = 1; i < 8; ++i) {
            dw += sw[i][lane];
            db += sb[i][lane];
        }
        if (a.dweight) store_any(a.dweight, a.p_dtype, c, dw);
        if (a.dbias) store_any(a.dbias, a.p_dtype, c, db);
    }
}

// f(TX{}, TY{}): y has x's type or float32.
template <typename F>
cudaError_t with_xy(const NormArgs &a, F &&f)
{
    return with_dtype(a.x_dtype, [&](auto tx) {
        if (a.y_dtype == HISS_F32) return f(tx, float{});
        return f(tx, tx);
    });
}

}  // namespace

cudaError_t layer_norm(const NormArgs &a, cudaStream_t s, int64_t *launches)
{
    return with_xy(a, [&](auto tx, auto ty) {
        k_norm<decltype(tx), decltype(ty)><<<(unsigned)a.n, kThreads, 0, s>>>(a);
        ++*launches;
        return cudaGetLastError();
    });
}

size_t layer_norm_grad_tmp_bytes(const NormArgs &) { return 0; }

cudaError_t layer_norm_grad(const NormArgs &a, void *, cudaStream_t s, int64_t *launches)
{
    return with_xy(a, [&](auto tx, auto ty) {
        if (a.dx && a.n > 0) {
            k_norm_dx<decltype(tx), decltype(ty)><<<(unsigned)a.n, kThreads, 0, s>>>(a);
            ++*launches;
        }
        if (a.dweight || a.dbias) {
            k_norm_dparam<decltype(tx), decltype(ty)><<<(unsigned)((a.width + 31) / 32), kThreads, 0, s>>>(a);
            ++*launches;
        }
        return cudaGetLastError();
    });
}

}  // namespace hiss
