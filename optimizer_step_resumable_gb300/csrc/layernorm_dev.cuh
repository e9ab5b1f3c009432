// layernorm_dev.cuh -- the layout of rows over threads that the forward and
// the backward pass share.
//
// A row is held by one group of kGroup threads (8, 16 or 32 lanes of a warp,
// or a whole block of 128 and more), each with up to kVecs vectors of 16
// bytes.  Vectors are cut at 16-byte boundaries of the address, not of the
// row: a row of any width at any place is a head of up to kE - 1 elements, a
// body of whole vectors, and a tail of up to kE - 1 elements; head and tail
// are one more element for each of 16 lanes.  Groups step through the rows
// by a multiple of 8, so the head's length -- which has at most 8 values over
// the rows -- is the same for all rows of a group, and a thread keeps the
// same columns, their weights and their gradient sums in registers
// throughout.
//
// Rows come through a ring in shared memory (cp.async).  How many bytes are
// on their way matters in both directions: too few leave the memory idle, too
// many make it jump between rows.  65536 x 4096 bf16 on GB300: forward 171 and
// 187 us with a ring of 64 and 96 KB an SM; backward 280 and 242 with 64 and
// 96, and 315 with 192 in twice the blocks.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "early_dev.cuh"
#include "layernorm.h"
#include "packed_dev.cuh"

namespace osr {
namespace ln {

using packed::add2;
using packed::both;
using packed::fma2;
using packed::mul2;

template <typename T>
constexpr int kE = 16 / int(sizeof(T));  // elements of a vector
template <typename T>
constexpr int kP = kE<T> / 2;  // pairs of a vector
constexpr int kRowStep = 8;    // groups step by a multiple of this: of kE for every type

__device__ __forceinline__ void widen(uint4 q, float2 (&f)[2])  // float32
{
    f[0] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
    f[1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
}
template <typename T>
__device__ __forceinline__ void widen16(uint4 q, float2 (&f)[4])  // 16-bit types
{
    const T* const t = nullptr;
    f[0] = detail::widen2(q.x, t);
    f[1] = detail::widen2(q.y, t);
    f[2] = detail::widen2(q.z, t);
    f[3] = detail::widen2(q.w, t);
}
template <typename T>
__device__ __forceinline__ void widen_as(uint4 q, float2 (&f)[kP<T>])
{
    if constexpr (sizeof(T) == 4)
        widen(q, f);
    else
        widen16<T>(q, f);
}
template <typename T>
__device__ __forceinline__ uint4 narrow_as(const float2 (&f)[kP<T>])
{
    if constexpr (sizeof(T) == 4) {
        return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y),
                          __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    } else {
        const T* const t = nullptr;
        return make_uint4(detail::pack2(f[0].x, f[0].y, t), detail::pack2(f[1].x, f[1].y, t),
                          detail::pack2(f[2].x, f[2].y, t), detail::pack2(f[3].x, f[3].y, t));
    }
}
template <int kPairs>
__device__ __forceinline__ void clear(float2 (&f)[kPairs])
{
#pragma unroll
    for (int p = 0; p < kPairs; ++p)
        f[p] = make_float2(0.0f, 0.0f);
}

__device__ __forceinline__ void store_one(float* p, float f) { *p = f; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float f) { *p = __float2bfloat16_rn(f); }
__device__ __forceinline__ void store_one(__half* p, float f) { *p = __float2half_rn(f); }

// Elements from p to the next 16-byte boundary.
template <typename T>
__device__ __forceinline__ int head_of(const T* p)
{
    return int((0 - reinterpret_cast<uintptr_t>(p) / sizeof(T)) & (kE<T> - 1));
}

// How the rows lie.  kFull: they fill the group's vectors, each at a 16-byte
// boundary.  kAligned: they end before the last of them.  kRagged: anywhere,
// but those of all arrays alike (mod 16 bytes).  kShifted: the output is cut
// elsewhere than x; it is cut anew in shared memory.  kMixed: dy too, which
// then is read element by element.
enum Rows { kFull, kAligned, kRagged, kShifted, kMixed };
static_assert(kMixed < kLnRows, "a place in LnBlocks for each");

// Which columns a thread holds: vectors at column(v) = start + v kStride, and
// (from kRagged on) one element of the head or the tail at edge, or -1.
template <typename T, int kGroup, Rows kRows>
struct Columns {
    static constexpr int kStride = kGroup * kE<T>;
    int lane, start, end, edge = -1;

    // row: any row of the group
    __device__ __forceinline__ Columns(int cols, int lane_, const T* row) : lane(lane_)
    {
        int head = 0;
        end = cols;
        if constexpr (kRows >= kRagged) {
            head = head_of(row);
            head = head < cols ? head : cols;
            const int body = (cols - head) / kE<T> * kE<T>;
            const int tail = cols - head - body;
            end = head + body;
            if (lane < 8)
                edge = lane < head ? lane : -1;
            else if (lane < 16)
                edge = lane - 8 < tail ? end + lane - 8 : -1;
        }
        start = head + lane * kE<T>;
    }
    __device__ __forceinline__ int column(int v) const { return start + v * kStride; }
    __device__ __forceinline__ bool has(int v) const { return kRows == kFull || column(v) < end; }
    __device__ __forceinline__ bool has_edge() const { return kRows >= kRagged && edge >= 0; }
};

// Whether p lies at a vector's boundary; known but for kMixed.
template <Rows kRows, typename T>
__device__ __forceinline__ bool is_cut(const T* p)
{
    return kRows != kMixed || (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// A vector at p, 16-byte aligned or (kMixed) not.
template <Rows kRows, typename T>
__device__ __forceinline__ void load_vec(const T* p, bool aligned, float2 (&f)[kP<T>])
{
    if (kRows != kMixed || aligned) {
        widen_as<T>(__ldg(reinterpret_cast<const uint4*>(p)), f);
    } else {
#pragma unroll
        for (int i = 0; i < kP<T>; ++i)
            f[i] = make_float2(detail::load1(p + 2 * i), detail::load1(p + 2 * i + 1));
    }
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, uint4 q)
{
    __stcs(reinterpret_cast<uint4*>(p), q);
}
// The elements [lo, hi) of a vector, at p.
__device__ __forceinline__ void store_some(float* p, uint4 q, int lo, int hi)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i >= lo && i < hi)
            p[i] = __uint_as_float(w[i]);
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, uint4 q, int lo, int hi)  // 16-bit types
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i >= lo && i < hi)
            reinterpret_cast<uint16_t*>(p)[i] = uint16_t(w[i / 2] >> (16 * (i & 1)));
}
// The vector that starts `bytes` (below 16, a multiple of an element) into a
// and ends in b.
template <typename T>
__device__ __forceinline__ uint4 joined(uint4 a, uint4 b, int bytes)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i)
        w[i] = bytes & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i)
        w[i] = bytes & 4 ? w[i + 1] : w[i];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (bytes & 2));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One weight (or bias); `none` where there is no array.
template <typename T>
__device__ __forceinline__ float weight_at(const void* w, bool f32, int c, float none)
{
    return !w    ? none
           : f32 ? __ldg(static_cast<const float*>(w) + c)
                 : detail::load1(static_cast<const T*>(w) + c);
}
// A thread's weights for the vector at column c.
template <typename T>
__device__ __forceinline__ void load_weights(const void* w, bool f32, int c, bool has, float none,
                                             float2 (&f)[kP<T>])
{
    const char* const at = static_cast<const char*>(w) + int64_t(c) * (f32 ? 4 : int(sizeof(T)));
    if (!w || !has) {
#pragma unroll
        for (int p = 0; p < kP<T>; ++p)
            f[p] = both(none);
    } else if (reinterpret_cast<uintptr_t>(at) & 15u) {
#pragma unroll
        for (int p = 0; p < kP<T>; ++p)
            f[p] = make_float2(weight_at<T>(w, f32, c + 2 * p, none),
                               weight_at<T>(w, f32, c + 2 * p + 1, none));
    } else if (f32) {
#pragma unroll
        for (int p = 0; p < kP<T>; p += 2) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(at) + p / 2);
            f[p] = make_float2(q.x, q.y);
            f[p + 1] = make_float2(q.z, q.w);
        }
    } else {
        widen_as<T>(__ldg(reinterpret_cast<const uint4*>(at)), f);
    }
}

// A thread's vectors of kStages rows of kArrays arrays, on their way through
// shared memory: every thread copies what it will read itself, so it waits
// for its own copies only and no barrier is needed.
template <typename T, int kThreads, int kVecs, int kArrays, int kStages>
struct Ring {
    static constexpr int kDepth = kStages, kVectors = kVecs;
    static constexpr int kBytes = kStages * kArrays * kVecs * kThreads * 16;
    uint4* base;

    __device__ __forceinline__ uint4* at(int stage, int array, int vec) const
    {
        return base + ((stage * kArrays + array) * kVecs + vec) * kThreads + threadIdx.x;
    }
    __device__ __forceinline__ void copy(int stage, int array, int vec, const T* from) const
    {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         uint32_t(__cvta_generic_to_shared(at(stage, array, vec)))),
                     "l"(from)
                     : "memory");
    }
    __device__ __forceinline__ void read(int stage, int array, int vec, float2 (&f)[kP<T>]) const
    {
        widen_as<T>(*at(stage, array, vec), f);
    }
};
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void wait_copies()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// Stages for about `want` bytes of ring per SM, 2 to `most` where they fit.
constexpr int stages_for(int stage_bytes, int blocks, int want, int most)
{
    const int fit = 208 * 1024 / blocks / stage_bytes;
    int n = want / blocks / stage_bytes;
    n = n < 2 ? 2 : n > most ? most : n;
    n = n > fit ? fit : n;
    return n < 1 ? 1 : n;
}

// The sums of kCount values over a group, in a fixed order, in every thread.
// `slots` (groups of a block): the warps' sums, two sets used in turn, so that
// one barrier per call is enough.
template <int kGroup, int kCount, int kMost>
__device__ __forceinline__ void group_sum(float (&s)[kCount], float (&slots)[2][kMost][16],
                                          int& turn)
{
    static_assert(kCount <= kMost, "a slot for each sum");
    constexpr int kLanes = kGroup < 32 ? kGroup : 32;
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < kCount; ++i)
            s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
    if constexpr (kGroup > 32) {
#pragma unroll
        for (int i = 0; i < kCount; ++i)
            if ((threadIdx.x & 31) == 0)
                slots[turn][i][threadIdx.x >> 5] = s[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            s[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < kGroup / 32; ++w)
                s[i] += slots[turn][i][w];
        }
        turn ^= 1;
    }
}

// The statistics of a row from a first mean and, of the differences d from it,
// their sum and the sum of their squares.  The first mean errs by up to a few
// 2^-24 of mean |x|, which moves every difference and adds its square to the
// variance.  Where that is much beside the spread the differences are exact,
// and their mean e is what the first mean lacks.  Elsewhere e is the rounding
// of the differences, below 2^-24 of the spread, where the first mean may be
// exact (sums of 16-bit values often are): an e below 2^-22 of the spread
// counts for nothing.  xhat = d rstd + shift.
struct Statistics {
    float mean, rstd, shift;
};
__device__ __forceinline__ Statistics statistics_of(float mean, const float (&d)[2], float inv,
                                                    float eps)
{
    const float square = d[1] * inv;
    float e = d[0] * inv;
    float var = __fmaf_rn(-e, e, square);
    if (!(e * e > 0x1p-44f * var)) {  // also where the sums are no numbers
        e = 0.0f;
        var = square;
    }
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn((var < 0.0f ? 0.0f : var) + eps));
    return Statistics{mean + e, rstd, -e * rstd};
}

template <int kGroup>
__device__ __forceinline__ void group_barrier()
{
    if constexpr (kGroup > 32)
        __syncthreads();
    else
        __syncwarp();
}

// A row of the output whose vectors are not x's: every thread has
// put its vectors into array 0 of the ring's stage, and each now takes the
// vector of `out` that starts `shift` elements into its own and ends in the
// next; what is left at the two ends goes element by element.  (Rows 1034
// apart into rows 1021 apart, 32768 x 1021 bf16, all of it element by element
// and this way: 73 and 39 us forward, 68 and 66 backward; 8192 x 8189: 211
// and 71, 223 and 153.)
// out: this thread's first vector.
template <typename T, int kGroup, Rows kRows, typename R>
__device__ __forceinline__ void store_shifted(const Columns<T, kGroup, kRows>& at, const R& ring,
                                              int stage, T* out, int shift)
{
#pragma unroll
    for (int v = 0; v < R::kVectors; ++v) {
        if (!at.has(v))
            continue;
        T* const p = out + v * at.kStride;
        const uint4 q = *ring.at(stage, 0, v);
        if (at.column(v) + kE<T> < at.end) {
            const uint4* const next = at.lane + 1 < kGroup ? ring.at(stage, 0, v) + 1
                                                           : ring.at(stage, 0, v + 1) + 1 - kGroup;
            store_vec(p + shift, joined<T>(q, *next, shift * int(sizeof(T))));
        } else {
            store_some(p, q, shift, kE<T>);
        }
        if (v == 0 && at.lane == 0)
            store_some(p, q, 0, shift);
    }
}

// Rows that do not fit a block's registers: a block looks at a row several
// times, the later ones from L2.  4096 x 32768 bf16, weights too, takes 195 us
// forward and 422 backward, 8192 x 16392 224 and 440 (element by element the
// first took 395 and 887).  Rows spread over clusters of blocks, held in
// registers, took 227 and 387 (303 and 481): each row waits for the cluster's
// barriers.
constexpr int kWideThreads = 512;
template <typename T>
using WideColumns = Columns<T, kWideThreads, kMixed>;

// A vector as it lies in memory.
template <typename T>
__device__ __forceinline__ uint4 load_raw(const T* p, bool aligned)
{
    if (aligned)
        return __ldg(reinterpret_cast<const uint4*>(p));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
        } else {
            const uint16_t* const h = reinterpret_cast<const uint16_t*>(p) + 2 * i;
            w[i] = uint32_t(__ldg(h)) | uint32_t(__ldg(h + 1)) << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Calls f(v, vectors) for a thread's vectors of a row of each array, kAtOnce
// of them on their way; p...: where its first lies.
template <typename T, int kAtOnce, typename C, typename F, typename... P>
__device__ __forceinline__ void each_vector(const C& at, F f, const P*... p)
{
    constexpr int kArrays = sizeof...(P);
    const T* const from[kArrays] = {p...};
    for (int v = 0; at.has(v); v += kAtOnce) {
        uint4 q[kAtOnce][kArrays];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
            if (at.has(v + u)) {
#pragma unroll
                for (int i = 0; i < kArrays; ++i)
                    q[u][i] = load_raw(from[i] + (v + u) * C::kStride, is_cut<kMixed>(from[i]));
            }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
            if (at.has(v + u)) {
                float2 x[kArrays][kP<T>];
#pragma unroll
                for (int i = 0; i < kArrays; ++i)
                    widen_as<T>(q[u][i], x[i]);
                f(v + u, x);
            }
    }
}
template <typename T>
__device__ __forceinline__ void store_any(T* p, bool aligned, uint4 q)
{
    if (aligned)
        store_vec(p, q);
    else
        store_some(p, q, 0, kE<T>);
}

// Threads of a block that holds such groups.
template <int kGroup>
constexpr int kBlockThreads = kGroup > 32 ? kGroup : 256;

// Calls f(Layout<kGroup, kUnits>) for rows of cols elements, cols <=
// kLnRegisterCols: kUnits x 8 elements a thread.
template <int G, int U>
struct Layout {
    static constexpr int kGroup = G, kUnits = U;
};
template <typename F>
int with_layout(int cols, bool aligned, F f)
{
    if (cols <= 64 && aligned) return f(Layout<8, 1>());  // no lanes for head and tail
    if (cols <= 128) return f(Layout<16, 1>());
    if (cols <= 256) return f(Layout<32, 1>());
    if (cols <= 512) return f(Layout<32, 2>());
    if (cols <= 768) return f(Layout<32, 3>());
    if (cols <= 1024) return f(Layout<32, 4>());
    if (cols <= 2048) return f(Layout<128, 2>());
    if (cols <= 4096) return f(Layout<128, 4>());
    if (cols <= 6144) return f(Layout<256, 3>());
    if (cols <= 8192) return f(Layout<256, 4>());
    return f(Layout<512, 4>());
}

// Resident blocks of a kernel per SM of the current device, which is allowed
// its shared memory there first.  Only an answer is kept in `known`.
template <typename F>
inline cudaError_t resident_blocks(F* kernel, int threads, int smem, std::atomic<int>& known,
                                   int* per_sm)
{
    int n = known.load(std::memory_order_relaxed);
    if (n == 0) {
        cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
        if (e == cudaSuccess && n < 1)
            return cudaErrorLaunchOutOfResources;
        if (e != cudaSuccess) {
            cudaGetLastError();  // returned here, not by a later call
            return e;
        }
        known.store(n, std::memory_order_relaxed);
    }
    *per_sm = n;
    return cudaSuccess;
}

// Blocks for `rows` rows, of `most` at once: the groups step by a multiple of
// kRowStep.
inline int64_t row_blocks(int64_t rows, int groups_per_block, int64_t most)
{
    const int unit = groups_per_block < kRowStep ? kRowStep / groups_per_block : 1;
    int64_t blocks = detail::ceil_div(rows, groups_per_block);
    blocks = detail::ceil_div(blocks, unit) * unit;
    most = most / unit * unit;
    return blocks > most ? (most < unit ? unit : most) : blocks;
}

// Whether every row of an array starts at a 16-byte boundary.
inline bool rows_aligned(const void* p, int64_t stride, size_t size)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && uint64_t(stride) * size % 16 == 0;
}
// Whether the rows of two arrays lie alike, mod 16 bytes.
inline bool rows_alike(const void* p, int64_t p_stride, const void* q, int64_t q_stride, size_t size)
{
    return (reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(q)) % 16 == 0 &&
           (uint64_t(p_stride) - uint64_t(q_stride)) * size % 16 == 0;
}

}  // namespace ln
}  // namespace osr
