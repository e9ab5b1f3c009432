// linear_dev.cuh -- what becomes of a sum of products before it is stored:
// bias, activation, residual, type.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "linear.h"

namespace osr {
namespace detail {

__device__ __forceinline__ float widen16(uint32_t bits, bool bf16)
{
    return bf16 ? __uint_as_float(bits << 16)
                : __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}
__device__ __forceinline__ uint16_t narrow16(float x, bool bf16)
{
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x))
                : __half_as_ushort(__float2half_rn(x));
}
__device__ __forceinline__ uint32_t narrow32(float lo, float hi, bool bf16)
{
    if (bf16) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&p);
    }
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ float load_as(const void* p, int64_t i, int32_t dtype)
{
    return dtype == ADAMW_DTYPE_F32
               ? static_cast<const float*>(p)[i]
               : widen16(static_cast<const uint16_t*>(p)[i], dtype == ADAMW_DTYPE_BF16);
}
__device__ __forceinline__ void store_as(void* p, int64_t i, int32_t dtype, float x)
{
    if (dtype == ADAMW_DTYPE_F32)
        static_cast<float*>(p)[i] = x;
    else
        static_cast<uint16_t*>(p)[i] = narrow16(x, dtype == ADAMW_DTYPE_BF16);
}
// 32 bytes of global memory.
__device__ __forceinline__ void load32(const void* p, uint32_t (&v)[8])
{
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                   "=r"(v[6]), "=r"(v[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// 1 / (1 + e^-x).  For x below -87 e^-x overflows and the quotient is 0, as
// the value is to float32's range.
__device__ __forceinline__ float logistic(float x)
{
    return __fdividef(1.0f, 1.0f + __expf(-x));
}

constexpr float kGeluScale = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

template <int kAct>
__device__ __forceinline__ float activated(float z)
{
    if constexpr (kAct == LINEAR_RELU)
        return z < 0.0f ? 0.0f : z;  // a NaN stays one
    else if constexpr (kAct == LINEAR_GELU)
        return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    else if constexpr (kAct == LINEAR_GELU_TANH)
        // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
        return z * logistic(2.0f * kGeluScale * (z + kGeluCube * z * z * z));
    else if constexpr (kAct == LINEAR_SILU)
        return z * logistic(z);
    else
        return z;
}

// The derivative of activated() at z.
template <int kAct>
__device__ __forceinline__ float slope(float z)
{
    if constexpr (kAct == LINEAR_RELU)
        return z > 0.0f ? 1.0f : 0.0f;
    else if constexpr (kAct == LINEAR_GELU)
        return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) +
               z * (0.39894228040143268f * __expf(-0.5f * z * z));
    else if constexpr (kAct == LINEAR_GELU_TANH) {
        const float g = logistic(2.0f * kGeluScale * (z + kGeluCube * z * z * z));
        const float t = g * (1.0f - g);  // 0 for large |z|, whose square may overflow
        return t > 0.0f ? g + z * (2.0f * kGeluScale) * t * (1.0f + 3.0f * kGeluCube * z * z)
                        : g;
    } else if constexpr (kAct == LINEAR_SILU) {
        const float g = logistic(z);
        return g * (1.0f + z * (1.0f - g));
    } else
        return 1.0f;
}

template <typename F>
__device__ __forceinline__ void with_activation(int32_t act, F&& f)
{
    switch (act) {
    case LINEAR_RELU: f(std::integral_constant<int, LINEAR_RELU>()); break;
    case LINEAR_GELU: f(std::integral_constant<int, LINEAR_GELU>()); break;
    case LINEAR_GELU_TANH: f(std::integral_constant<int, LINEAR_GELU_TANH>()); break;
    case LINEAR_SILU: f(std::integral_constant<int, LINEAR_SILU>()); break;
    default: f(std::integral_constant<int, LINEAR_NONE>());
    }
}

// One element, from its sum to memory.
template <int kAct>
__device__ __forceinline__ void finish_one(const LinearOut& o, int64_t row, int64_t column,
                                           float sum)
{
    float z = sum * o.alpha;
    if (o.bias)
        z += load_as(o.bias, column, o.bias_dtype);
    if (o.z)
        store_as(o.z, row * o.z_stride + column, o.dtype, z);
    float y = activated<kAct>(z);
    if (o.residual)
        y += load_as(o.residual, row * o.residual_stride + column, o.residual_dtype);
    const int64_t at = row * o.stride + column;
    if (o.accumulate)
        y += load_as(o.out, at, o.dtype);
    store_as(o.out, at, o.dtype, y);
}

}  // namespace detail
}  // namespace osr
