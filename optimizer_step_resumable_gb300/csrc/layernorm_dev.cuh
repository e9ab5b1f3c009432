// layernorm_dev.cuh -- the layout of rows over threads that the forward and
// the backward pass share.
//
// A row is held in the registers of one group of kGroup threads (8, 16 or 32
// lanes of a warp, or a whole block of 128 and more), each with up to kVecs
// vectors of 8 adjacent elements.  Vectors are cut at multiples of 8
// elements of the address, not of the row: a row of any width at any place
// is read in 16-byte (32-byte for float32) accesses but for its first and
// last vector.  The vectors start `off` elements before the row, off in
// 0..7.  Groups step through the rows by a multiple of 8, so off -- which
// has at most 8 values over the rows -- is the same for all rows of a group,
// and a thread keeps the same columns, their weights and their gradient sums
// in registers throughout.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "layernorm.h"

namespace osr {
namespace ln {

constexpr int kE = 8;  // elements of a vector

// 8 adjacent elements as they lie in memory.
template <typename T>
struct Raw {  // 16-bit types
    uint4 q;
};
template <>
struct Raw<float> {
    float4 a, b;
};

template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p)
{
    return Raw<T>{__ldcs(reinterpret_cast<const uint4*>(p))};
}
template <>
__device__ __forceinline__ Raw<float> load_raw<float>(const float* p)
{
    const float4* q = reinterpret_cast<const float4*>(p);
    return Raw<float>{__ldcs(q), __ldcs(q + 1)};
}

__device__ __forceinline__ void pair(uint32_t u, float& lo, float& hi, const __nv_bfloat16*)
{
    lo = __uint_as_float(u << 16);
    hi = __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ void pair(uint32_t u, float& lo, float& hi, const __half*)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
    lo = f.x;
    hi = f.y;
}
template <typename T>
__device__ __forceinline__ void widen(const Raw<T>& r, float (&f)[kE])
{
    pair(r.q.x, f[0], f[1], static_cast<const T*>(nullptr));
    pair(r.q.y, f[2], f[3], static_cast<const T*>(nullptr));
    pair(r.q.z, f[4], f[5], static_cast<const T*>(nullptr));
    pair(r.q.w, f[6], f[7], static_cast<const T*>(nullptr));
}
template <>
__device__ __forceinline__ void widen<float>(const Raw<float>& r, float (&f)[kE])
{
    f[0] = r.a.x, f[1] = r.a.y, f[2] = r.a.z, f[3] = r.a.w;
    f[4] = r.b.x, f[5] = r.b.y, f[6] = r.b.z, f[7] = r.b.w;
}

__device__ __forceinline__ uint32_t pack(float lo, float hi, const __nv_bfloat16*)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack(float lo, float hi, const __half*)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[kE])
{
    const T* t = nullptr;
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack(f[0], f[1], t), pack(f[2], f[3], t),
                                                   pack(f[4], f[5], t), pack(f[6], f[7], t)));
}
template <>
__device__ __forceinline__ void store_vec<float>(float* p, const float (&f)[kE])
{
    float4* q = reinterpret_cast<float4*>(p);
    __stcs(q, make_float4(f[0], f[1], f[2], f[3]));
    __stcs(q + 1, make_float4(f[4], f[5], f[6], f[7]));
}

__device__ __forceinline__ void store_one(float* p, float f) { *p = f; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float f) { *p = __float2bfloat16_rn(f); }
__device__ __forceinline__ void store_one(__half* p, float f) { *p = __float2half_rn(f); }

// How many elements p lies past a vector's boundary.
template <typename T>
__device__ __forceinline__ int offset_of(const T* p)
{
    return int((reinterpret_cast<uintptr_t>(p) / sizeof(T)) & (kE - 1));
}

// A thread's vector starting at column c of a row, c0 = -off .. cols - 1.
// kRagged: the vector may hang over either end of the row, and `whole` says
// whether this array's rows are cut at the same places; elements outside the
// row read as 0 and are not written.
template <bool kRagged, typename T>
__device__ __forceinline__ void load8(const T* row, int c, int cols, bool whole, float (&f)[kE])
{
    if (!kRagged || (whole && c >= 0 && c + kE <= cols)) {
        if (!kRagged && c >= cols) {
#pragma unroll
            for (int i = 0; i < kE; ++i)
                f[i] = 0.0f;
            return;
        }
        widen<T>(load_raw<T>(row + c), f);
    } else {
#pragma unroll
        for (int i = 0; i < kE; ++i)
            f[i] = c + i >= 0 && c + i < cols ? detail::load1(row + c + i) : 0.0f;
    }
}
template <bool kRagged, typename T>
__device__ __forceinline__ void store8(T* row, int c, int cols, bool whole, const float (&f)[kE])
{
    if (!kRagged || (whole && c >= 0 && c + kE <= cols)) {
        if (kRagged || c < cols)
            store_vec<T>(row + c, f);
    } else {
#pragma unroll
        for (int i = 0; i < kE; ++i)
            if (c + i >= 0 && c + i < cols)
                store_one(row + c + i, f[i]);
    }
}

// Whether element i of a thread's vector at column c lies in the row.
template <bool kRagged>
__device__ __forceinline__ bool in_row(int c, int i, int cols)
{
    return kRagged ? (c + i >= 0 && c + i < cols) : c < cols;
}

// A thread's weights (or biases) for one of its vectors; `none` where there
// is no array and outside the row.
template <typename T>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int c, int cols, float none,
                                            float (&f)[kE])
{
#pragma unroll
    for (int i = 0; i < kE; ++i) {
        const bool in = w && c + i >= 0 && c + i < cols;
        f[i] = !in   ? none
               : f32 ? static_cast<const float*>(w)[c + i]
                     : detail::load1(static_cast<const T*>(w) + c + i);
    }
}

// The sums of a and b over a group, in a fixed order, in every thread.
// `slots`: for groups of a block, 2 x (kGroup / 32) float2 in shared memory,
// used in turn, so that one barrier per sum is enough.
template <int kGroup>
__device__ __forceinline__ float2 group_sum(float a, float b, float2 (*slots)[32], int& turn)
{
    constexpr int kLanes = kGroup < 32 ? kGroup : 32;
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, d);
        b += __shfl_xor_sync(0xffffffffu, b, d);
    }
    if constexpr (kGroup > 32) {
        if ((threadIdx.x & 31) == 0)
            slots[turn][threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int w = 0; w < kGroup / 32; ++w) {
            const float2 s = slots[turn][w];
            a += s.x;
            b += s.y;
        }
        turn ^= 1;
    }
    return make_float2(a, b);
}

// Threads of a block that holds such groups.
template <int kGroup>
constexpr int kBlockThreads = kGroup > 32 ? kGroup : 256;

// Calls f(Layout<kGroup, kVecs>) for the layout of rows that span `span`
// columns (cols, or cols + 7 where rows may start between boundaries); span
// <= kLnRegisterCols.
template <int G, int V>
struct Layout {
    static constexpr int kGroup = G, kVecs = V;
};
template <typename F>
int with_layout(int span, F f)
{
    if (span <= 64) return f(Layout<8, 1>());
    if (span <= 128) return f(Layout<16, 1>());
    if (span <= 256) return f(Layout<32, 1>());
    if (span <= 512) return f(Layout<32, 2>());
    if (span <= 768) return f(Layout<32, 3>());
    if (span <= 1024) return f(Layout<32, 4>());
    if (span <= 2048) return f(Layout<128, 2>());
    if (span <= 4096) return f(Layout<128, 4>());
    if (span <= 8192) return f(Layout<256, 4>());
    return f(Layout<512, 4>());
}

// Whether every row of an array starts at a vector's boundary.
template <typename T>
inline bool rows_aligned(const void* p, int64_t stride)
{
    return reinterpret_cast<uintptr_t>(p) % (kE * sizeof(T)) == 0 && stride % kE == 0;
}

}  // namespace ln
}  // namespace osr
