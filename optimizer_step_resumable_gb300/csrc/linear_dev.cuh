// linear_dev.cuh -- what becomes of a sum of products before it is stored:
// bias, activation, residual, type.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "linear.h"
#include "packed_dev.cuh"

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

// 32 rows of 64 16-bit elements on their way from a warp's lanes, a row each,
// to memory: through 4 KB of shared memory, so that eight lanes write the 128
// bytes of a row (the cross entropy's backward pass 773 us with each lane writing
// its own row, 32 bytes at a time, 765 so).  16-byte pieces lie swizzled, at piece
// XOR row, so that neither way meets a bank twice.
__device__ __forceinline__ void strip_put(uint4* strip, int piece, uint4 w)
{
    const int lane = threadIdx.x % 32;
    strip[8 * lane + (piece ^ (lane & 7))] = w;
}
// `to`: the first row's first element, rows `stride` elements apart, `count` of
// them and `columns` (a multiple of 8) of each written.
__device__ __forceinline__ void strip_write(const uint4* strip, uint16_t* to, int64_t stride,
                                            int32_t count, int32_t columns)
{
    const int lane = threadIdx.x % 32, piece = lane % 8;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const int r = i + lane / 8;
        const uint4 w = strip[8 * r + (piece ^ (r & 7))];
        if (r < count && 8 * piece < columns)
            *reinterpret_cast<uint4*>(to + r * stride + 8 * piece) = w;
    }
    __syncwarp();
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

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 exp2_fast(float2 x)
{
    return make_float2(exp2_fast(x.x), exp2_fast(x.y));
}
__device__ __forceinline__ float2 inverse_fast(float2 x)
{
    float2 y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(x.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(x.y));
    return y;
}
__device__ __forceinline__ float2 minus_abs(float2 z)
{
    return make_float2(-fabsf(z.x), -fabsf(z.y));
}
// The larger and the smaller, of which a NaN stays one.
__device__ __forceinline__ float2 at_least(float2 z, float a)
{
    float2 y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y.x) : "f"(z.x), "f"(a));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y.y) : "f"(z.y), "f"(a));
    return y;
}
__device__ __forceinline__ float2 at_most(float2 z, float a)
{
    float2 y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y.x) : "f"(z.x), "f"(a));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y.y) : "f"(z.y), "f"(a));
    return y;
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kGeluScale = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;
// Beyond +-kFar every activation here is z or 0 to float32, and every slope 1
// or 0; what would multiply an infinity by 0 takes z no further.
constexpr float kFar = 100.0f;

// 1 / (1 + 2^x): 0 where 2^x overflows.
__device__ __forceinline__ float2 logistic(float2 x)
{
    return inverse_fast(packed::add2(exp2_fast(x), packed::both(1.0f)));
}

// What gelu and its slope are made of, at x = min(|z|, kFar): e = e^(-x^2 / 2) and
// the normal distribution's tail beyond x, which is e R(x) with a smooth R: R = t
// P(t), t = 1 / (1 + 0.305 x), P the polynomial with the least relative error over 0
// <= x <= 14 and P(1) = 1/2 (a linear program): 1.1e-7, 4.1e-7 in float32.  Relative,
// since gelu below 0 is z times the tail: what bounds the tail's absolute error only
// leaves 4e-4 to 3e-2 of gelu between -3 and -12, more than the rounding to 16 bits.
// e itself errs by about x^2 2^-24, and is 0 beyond 13.2, where it is below 2^-126.  A
// power of two and a reciprocal, and products in pairs, where erfcf() takes some 40
// instructions an element.  That showed: the 32768 elements of a block's tile have
// 6000 cycles beside the products of 768 inputs.
struct Normal {
    float2 e, tail;
};
__device__ __forceinline__ Normal normal(float2 below)  // -x
{
    using namespace packed;
    const float2 t = inverse_fast(fma2(below, both(-0.305f), both(1.0f)));
    float2 p = fma2(t, both(0.036452897f), both(-0.15199922f));
    p = fma2(p, t, both(0.18407598f));
    p = fma2(p, t, both(-0.036524225f));
    p = fma2(p, t, both(0.1202834f));
    p = fma2(p, t, both(0.10363552f));
    p = fma2(p, t, both(0.12243386f));
    p = fma2(p, t, both(0.12164179f));
    const float2 e = exp2_fast(mul2(mul2(below, below), both(-0.5f * kLog2E)));
    return Normal{e, mul2(mul2(p, t), e)};
}

template <int kAct>
__device__ __forceinline__ float2 activated(float2 z)
{
    using namespace packed;
    if constexpr (kAct == LINEAR_RELU) {
        // a NaN stays one
        return make_float2(z.x < 0.0f ? 0.0f : z.x, z.y < 0.0f ? 0.0f : z.y);
    } else if constexpr (kAct == LINEAR_GELU) {
        // max(z, 0) - |z| (1 - distribution at |z|)
        const float2 below = at_least(minus_abs(z), -kFar);
        return fma2(below, normal(below).tail, at_least(z, 0.0f));
    } else if constexpr (kAct == LINEAR_GELU_TANH) {
        // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
        constexpr float k = -2.0f * kGeluScale * kLog2E;
        const float2 near = at_least(z, -kFar);
        const float2 w = fma2(mul2(near, near), both(k * kGeluCube), both(k));
        return mul2(near, logistic(mul2(near, w)));
    } else if constexpr (kAct == LINEAR_SILU) {
        const float2 near = at_least(z, -kFar);
        return mul2(near, logistic(mul2(near, both(-kLog2E))));
    } else {
        return z;
    }
}

// The derivative of activated() at z.
template <int kAct>
__device__ __forceinline__ float2 slope(float2 z)
{
    using namespace packed;
    if constexpr (kAct == LINEAR_RELU) {
        const auto one = [](float x) { return x > 0.0f ? 1.0f : x != x ? x : 0.0f; };
        return make_float2(one(z.x), one(z.y));
    }
    const float2 near = at_most(at_least(z, -kFar), kFar);
    if constexpr (kAct == LINEAR_GELU) {
        const Normal n = normal(minus_abs(near));
        const float2 rest = fma2(n.tail, both(-1.0f), both(1.0f));
        const float2 d = make_float2(near.x < 0.0f ? n.tail.x : rest.x,
                                     near.y < 0.0f ? n.tail.y : rest.y);
        return fma2(mul2(near, both(0.39894228040143268f)), n.e, d);
    } else if constexpr (kAct == LINEAR_GELU_TANH) {
        constexpr float k = -2.0f * kGeluScale * kLog2E;
        const float2 square = mul2(near, near);
        const float2 g = logistic(mul2(near, fma2(square, both(k * kGeluCube), both(k))));
        const float2 t = mul2(mul2(near, g), fma2(g, both(-1.0f), both(1.0f)));
        return fma2(t, fma2(square, both(6.0f * kGeluScale * kGeluCube), both(2.0f * kGeluScale)),
                    g);
    } else {
        const float2 g = logistic(mul2(near, both(-kLog2E)));
        return mul2(g, fma2(near, fma2(g, both(-1.0f), both(1.0f)), both(1.0f)));
    }
}

// act, or the products of g with its slopes, of N values.
template <int kAct, int N>
__device__ __forceinline__ void activate_all(float (&v)[N])
{
    if constexpr (kAct == LINEAR_NONE)
        return;
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
        const float2 y = activated<kAct>(make_float2(v[i], v[i + 1]));
        v[i] = y.x, v[i + 1] = y.y;
    }
    if constexpr (N % 2)
        v[N - 1] = activated<kAct>(make_float2(v[N - 1], 0.0f)).x;
}
template <int kAct, int N>
__device__ __forceinline__ void times_slopes(float (&g)[N], const float (&z)[N])
{
    static_assert(N % 2 == 0, "");
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 s = packed::mul2(make_float2(g[i], g[i + 1]),
                                      slope<kAct>(make_float2(z[i], z[i + 1])));
        g[i] = s.x, g[i + 1] = s.y;
    }
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

// With the factor that is on the device.
__device__ __forceinline__ LinearOut with_factor(const LinearOut& o)
{
    LinearOut r = o;
    if (o.alpha_factor)
        r.alpha *= *o.alpha_factor;
    return r;
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
    activate_all<kAct>(v);
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
