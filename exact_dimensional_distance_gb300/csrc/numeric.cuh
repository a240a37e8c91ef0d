// Element types of the operators on parameters and activations: conversions
// between float32, float16 and bfloat16 (round to nearest even) and the
// dispatch from hiss_dtype values to types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "hiss.h"

namespace hiss {

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

// Element i of an array of a type known at run time (parameters, read once per block).
__device__ __forceinline__ float load_any(const void *p, int dtype, int64_t i)
{
    if (dtype == HISS_F32) return static_cast<const float *>(p)[i];
    if (dtype == HISS_F16) return to_f32(static_cast<const __half *>(p)[i]);
    return to_f32(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void store_any(void *p, int dtype, int64_t i, float v)
{
    if (dtype == HISS_F32) static_cast<float *>(p)[i] = v;
    else if (dtype == HISS_F16) static_cast<__half *>(p)[i] = from_f32<__half>(v);
    else static_cast<__nv_bfloat16 *>(p)[i] = from_f32<__nv_bfloat16>(v);
}

}  // namespace hiss
