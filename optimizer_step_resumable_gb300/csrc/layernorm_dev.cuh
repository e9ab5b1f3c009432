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

__device__ __forceinline__ void store_one(float* p, float f) { *p = f; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float f) { *p = __float2bfloat16_rn(f); }
__device__ __forceinline__ void store_one(__half* p, float f) { *p = __float2half_rn(f); }

using detail::Raw8;
using detail::store8_cs;
using detail::widen8;

// How many elements p lies past a vector's boundary.
template <typename T>
__device__ __forceinline__ int offset_of(const T* p)
{
    return int((reinterpret_cast<uintptr_t>(p) / sizeof(T)) & (kE - 1));
}

// A thread's vector starts at column c of a row, c = -off .. cols - 1 or past
// the end.  kRagged: it may hang over either end of the row.  Elements outside
// the row count as 0 and are not written.
template <bool kRagged>
__device__ __forceinline__ bool is_full(int c, int cols)
{
    return kRagged ? c >= 0 && c + kE <= cols : c < cols;
}
template <typename T>
__device__ __forceinline__ void load_elements(const T* row, int c, int cols, float (&f)[kE])
{
#pragma unroll
    for (int i = 0; i < kE; ++i)
        f[i] = c + i >= 0 && c + i < cols ? detail::load1(row + c + i) : 0.0f;
}
// whole: this array's rows are cut where the vectors are.
template <bool kRagged, typename T>
__device__ __forceinline__ void store_vec(T* row, int c, int cols, bool whole, const float (&f)[kE])
{
    if (is_full<kRagged>(c, cols) && (!kRagged || whole)) {
        store8_cs(row + c, f);
    } else if (kRagged) {
#pragma unroll
        for (int i = 0; i < kE; ++i)
            if (c + i >= 0 && c + i < cols)
                store_one(row + c + i, f[i]);
    }
}

// A thread's vectors of kStages rows of kArrays arrays, on their way through
// shared memory (cp.async): every thread copies what it will read itself, so
// it waits for its own copies only and no barrier is needed.
template <typename T, int kThreads, int kVecs, int kArrays, int kStages>
struct Ring {
    static constexpr int kDepth = kStages;
    static constexpr int kHalves = int(sizeof(T)) / 2;  // 16-byte pieces of a vector
    static constexpr int kBytes = kStages * kArrays * kVecs * kHalves * kThreads * 16;
    uint4* base;

    __device__ __forceinline__ uint4* at(int stage, int array, int vec, int half) const
    {
        return base + (((stage * kArrays + array) * kVecs + vec) * kHalves + half) * kThreads +
               threadIdx.x;
    }
    __device__ __forceinline__ void copy(int stage, int array, int vec, const T* from) const
    {
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             uint32_t(__cvta_generic_to_shared(at(stage, array, vec, h)))),
                         "l"(reinterpret_cast<const char*>(from) + 16 * h)
                         : "memory");
    }
    __device__ __forceinline__ void read(int stage, int array, int vec, float (&f)[kE]) const
    {
        if constexpr (kHalves == 1) {
            widen8(Raw8<T>{*at(stage, array, vec, 0)}, f);
        } else {
            const float4 a = *reinterpret_cast<const float4*>(at(stage, array, vec, 0));
            const float4 b = *reinterpret_cast<const float4*>(at(stage, array, vec, 1));
            widen8(Raw8<float>{a, b}, f);
        }
    }
};
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void wait_copies()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// Stages that fit `blocks` resident blocks, at most 3.
constexpr int stages_for(int stage_bytes, int blocks)
{
    const int n = 208 * 1024 / blocks / stage_bytes;
    return n < 1 ? 1 : n > 3 ? 3 : n;
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

// Resident blocks of a kernel per SM, which is allowed its shared memory
// first.
template <typename F>
inline int resident_blocks(F* kernel, int threads, int smem)
{
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess)
        return 1;
    return n < 1 ? 1 : n;
}

// Whether every row of an array starts at a vector's boundary.
template <typename T>
inline bool rows_aligned(const void* p, int64_t stride)
{
    return reinterpret_cast<uintptr_t>(p) % (kE * sizeof(T)) == 0 && stride % kE == 0;
}

}  // namespace ln
}  // namespace osr
