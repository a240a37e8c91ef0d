// Element types of the operators on parameters and activations: conversions
// between float32, float16 and bfloat16 (round to nearest even), the dispatch
// from hiss_dtype values to types, and packs of elements that are read or
// written with one access.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "hiss.h"
#include "ptx.cuh"

namespace hiss {

constexpr int kSMs = 152;  // GB300

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// f(T{}) with T the element type of a hiss_dtype.
template <typename F>
cudaError_t with_dtype(int dtype, F &&f)
{
    if (dtype == HISS_F32) return f(float{});
    if (dtype == HISS_F16) return f(__half{});
    return f(__nv_bfloat16{});
}

inline size_t dtype_bytes(int dtype) { return dtype == HISS_F32 ? 4 : 2; }

// E elements in accesses of up to 16 bytes.
template <typename T, int E>
struct alignas(sizeof(T) * E < 16 ? sizeof(T) * E : 16) Pack {
    T v[E];
};

template <typename T, int E>
__device__ __forceinline__ Pack<T, E> load_pack(const T *p)
{
    return *reinterpret_cast<const Pack<T, E> *>(p);
}
template <typename T, int E>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, E> &v)
{
    *reinterpret_cast<Pack<T, E> *>(p) = v;
}

// Pairs of elements as float32 pairs, which the f32x2 instructions
// (__fadd2_rn, __fmul2_rn, __ffma2_rn: two round-to-nearest operations each) take.
__device__ __forceinline__ float2 pair_of(const float *p) { return make_float2(p[0], p[1]); }
__device__ __forceinline__ float2 pair_of(const __half *p)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(p));
}
__device__ __forceinline__ float2 pair_of(const __nv_bfloat16 *p)
{
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p));
}
__device__ __forceinline__ void set_pair(float *p, float2 v) { p[0] = v.x, p[1] = v.y; }
__device__ __forceinline__ void set_pair(__half *p, float2 v)
{
    *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(v.x, v.y);
}
__device__ __forceinline__ void set_pair(__nv_bfloat16 *p, float2 v)
{
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Asynchronous copy of a pack of whole 16-byte lines to shared memory.
template <typename T, int E>
__device__ __forceinline__ void copy_pack_async(Pack<T, E> *d, const T *p)
{
    constexpr int B = sizeof(T) * E;
    static_assert(B % 16 == 0, "whole lines");
#pragma unroll
    for (int i = 0; i < B; i += 16) cp_async16(reinterpret_cast<char *>(d) + i, reinterpret_cast<const char *>(p) + i);
}

// E consecutive parameters of a type known at run time (read once per block).
template <int E>
__device__ __forceinline__ void load_params(const void *p, int dtype, int64_t i, float (&v)[E])
{
    if (dtype == HISS_F32) {
        const auto k = load_pack<float, E>(static_cast<const float *>(p) + i);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = k.v[e];
    } else if (dtype == HISS_F16) {
        const auto k = load_pack<__half, E>(static_cast<const __half *>(p) + i);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = to_f32(k.v[e]);
    } else {
        const auto k = load_pack<__nv_bfloat16, E>(static_cast<const __nv_bfloat16 *>(p) + i);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = to_f32(k.v[e]);
    }
}
__device__ __forceinline__ float load_any(const void *p, int dtype, int64_t i)
{
    float v[1];
    load_params<1>(p, dtype, i, v);
    return v[0];
}
__device__ __forceinline__ void store_any(void *p, int dtype, int64_t i, float v)
{
    if (dtype == HISS_F32) static_cast<float *>(p)[i] = v;
    else if (dtype == HISS_F16) static_cast<__half *>(p)[i] = from_f32<__half>(v);
    else static_cast<__nv_bfloat16 *>(p)[i] = from_f32<__nv_bfloat16>(v);
}

// Whether rows of a matrix can be accessed E elements at a time.
inline bool rows_aligned(const void *p, int64_t stride, int dtype, int e)
{
    const size_t b = dtype_bytes(dtype) * e < 16 ? dtype_bytes(dtype) * e : 16;
    return reinterpret_cast<uintptr_t>(p) % b == 0 && (stride * dtype_bytes(dtype)) % b == 0;
}

// Lets a kernel use bytes of dynamic shared memory, once per device (done: a bit
// for each, of this kernel alone).
template <typename K>
cudaError_t allow_shared(K kernel, size_t bytes, std::atomic<uint64_t> &done)
{
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (device & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// ---- launches that overlap the kernel before them ---------------------------
// A kernel launched with launch_after may start while the kernel before it on
// the stream is finishing; it calls wait_for_previous before it touches
// anything that kernel writes.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, const A &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
__device__ __forceinline__ void wait_for_previous() { cudaGridDependencySynchronize(); }
// Lets the dependent kernel start launching (its wait still covers everything
// this kernel writes).
__device__ __forceinline__ void let_next_start() { cudaTriggerProgrammaticLaunchCompletion(); }

}  // namespace hiss
