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

// N elements from place i of p; whole: eight on a vector's boundary.
template <int N>
__device__ __forceinline__ void load_some(const void* p, int64_t i, int32_t dtype, bool whole,
                                          float (&v)[N])
{
    if constexpr (N == 8)
        if (whole) {
            if (dtype == ADAMW_DTYPE_F32) {
                uint32_t w[8];
                load32(static_cast<const float*>(p) + i, w);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = __uint_as_float(w[j]);
            } else {
                const uint4 q =
                    *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[2 * j] = widen16(w[j] & 0xFFFFu, dtype == ADAMW_DTYPE_BF16);
                    v[2 * j + 1] = widen16(w[j] >> 16, dtype == ADAMW_DTYPE_BF16);
                }
            }
            return;
        }
#pragma unroll
    for (int j = 0; j < N; ++j)
        v[j] = load_as(p, i + j, dtype);
}
template <int N>
__device__ __forceinline__ void store_some(void* p, int64_t i, int32_t dtype, bool whole,
                                           const float (&v)[N])
{
    if constexpr (N == 8)
        if (whole) {
            if (dtype == ADAMW_DTYPE_F32) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = __float_as_uint(v[j]);
                store32(static_cast<float*>(p) + i, w);
            } else {
                const bool bf16 = dtype == ADAMW_DTYPE_BF16;
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
                    make_uint4(narrow32(v[0], v[1], bf16), narrow32(v[2], v[3], bf16),
                               narrow32(v[4], v[5], bf16), narrow32(v[6], v[7], bf16));
            }
            return;
        }
#pragma unroll
    for (int j = 0; j < N; ++j)
        store_as(p, i + j, dtype, v[j]);
}

// 1 / (1 + e^-x).  For x below -87 e^-x overflows and the quotient is 0, as
// the value is to float32's range.
__device__ __forceinline__ float logistic(float x)
{
    return __fdividef(1.0f, 1.0f + __expf(-x));
}

// What gelu and its slope are made of: e = e^(-z^2 / 2) and the normal
// distribution at z, (1 + erf(z / sqrt 2)) / 2, by formula 7.1.26 of Abramowitz
// and Stegun's handbook, which is within 1.5e-7 of erf: one power of two and
// one reciprocal, where erff() takes some 40 instructions, which showed (a
// tile's 32768 elements have 6000 cycles beside the products of 768 inputs).
struct Normal {
    float e, below;
};
__device__ __forceinline__ Normal normal(float z)
{
    const float x = fabsf(z) * 0.70710678118654752f;
    const float t = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
    float p = fmaf(t, 1.061405429f, -1.453152027f);
    p = fmaf(p, t, 1.421413741f);
    p = fmaf(p, t, -0.284496736f);
    p = fmaf(p, t, 0.254829592f);
    const float e = __expf(-x * x), h = 0.5f * p * t * e;
    return Normal{e, z < 0.0f ? h : 1.0f - h};
}

constexpr float kGeluScale = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

template <int kAct>
__device__ __forceinline__ float activated(float z)
{
    if constexpr (kAct == LINEAR_RELU)
        return z < 0.0f ? 0.0f : z;  // a NaN stays one
    else if constexpr (kAct == LINEAR_GELU)
        return z * normal(z).below;
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
    else if constexpr (kAct == LINEAR_GELU) {
        const Normal n = normal(z);
        return fmaf(z * 0.39894228040143268f, n.e, n.below);
    } else if constexpr (kAct == LINEAR_GELU_TANH) {
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

// N neighbouring elements, from their sums to memory: one, or eight on a
// vector's boundary if the rows are on vectors.
template <int kAct, int N>
__device__ __forceinline__ void finish_some(const LinearOut& o, int64_t row, int64_t column,
                                            float (&v)[N])
{
    const bool whole = N == 8 && o.vectors;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] *= o.alpha;
        if (o.bias)
            v[i] += load_as(o.bias, column + i, o.bias_dtype);
    }
    if (o.z)
        store_some(o.z, row * o.z_stride + column, o.dtype, whole, v);
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = activated<kAct>(v[i]);
    if (o.residual) {
        float more[N];
        load_some(o.residual, row * o.residual_stride + column, o.residual_dtype, whole, more);
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] += more[i];
    }
    store_some(o.out, row * o.stride + column, o.dtype, whole, v);
}

}  // namespace detail
}  // namespace osr
