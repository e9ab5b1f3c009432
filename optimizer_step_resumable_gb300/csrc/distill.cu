// distill.cu -- loss and gradient of a student's logits against a teacher's
// top k.
//
// Both are bound by memory: the logits are read once (and their gradient
// written once).  A block has a row.  Forward, it keeps a running maximum and
// sum of exponentials, in powers of two; the k entries are a gather beside
// it.  Backward, p - q is p everywhere but at k places, so the row is written
// as p first and those places anew.
#include <cmath>

#include "distill.h"
#include "early_dev.cuh"
#include "linear_dev.cuh"

namespace osr {
namespace {

using namespace detail;

// Small blocks, many of them: what one waits for, others' loads fill (8192 x
// 32000 bf16 forward in blocks of 512 threads, each row's teacher read by all of
// them at the end: 154 us, against 80).
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kAtOnce = 4;  // vectors of a thread on their way
constexpr float kLn2 = 0.69314718055994531f;

// What exponentials are taken relative to: never -inf, of which the
// difference to itself is no number.
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.0f : m; }

template <typename T>
constexpr int kE = 16 / int(sizeof(T));
template <typename T>
constexpr bool kBf16 = std::is_same_v<T, __nv_bfloat16>;

template <typename T>
__device__ __forceinline__ float one(const T* p)
{
    if constexpr (sizeof(T) == 4)
        return *p;
    else
        return widen16(*reinterpret_cast<const uint16_t*>(p), kBf16<T>);
}
template <typename T>
__device__ __forceinline__ void put(T* p, float x)
{
    if constexpr (sizeof(T) == 4)
        *p = x;
    else
        *reinterpret_cast<uint16_t*>(p) = narrow16(x, kBf16<T>);
}
// The pairs of a vector.
template <typename T>
__device__ __forceinline__ float2 pair_of(const uint32_t (&w)[4], int i)
{
    if constexpr (sizeof(T) == 4)
        return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else if constexpr (kBf16<T>)
        return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
}
// A vector of -inf.
template <typename T>
__device__ __forceinline__ uint4 nothing()
{
    const uint32_t w = sizeof(T) == 4 ? 0xFF800000u : kBf16<T> ? 0xFF80FF80u : 0xFC00FC00u;
    return make_uint4(w, w, w, w);
}
// The largest element of `N` vectors; NaN are passed over, as by fmaxf.
template <typename T, int N>
__device__ __forceinline__ float largest(const uint4 (&q)[N])
{
    if constexpr (sizeof(T) == 4) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i)
            top = fmaxf(fmaxf(top, fmaxf(__uint_as_float(q[i].x), __uint_as_float(q[i].y))),
                        fmaxf(__uint_as_float(q[i].z), __uint_as_float(q[i].w)));
        return top;
    } else {
        using P = std::conditional_t<kBf16<T>, __nv_bfloat162, __half2>;
        const auto as = [](const uint32_t& w) { return *reinterpret_cast<const P*>(&w); };
        P top = as(q[0].x);
#pragma unroll
        for (int i = 0; i < N; ++i)
            top = __hmax2(__hmax2(top, __hmax2(as(q[i].x), as(q[i].y))),
                          __hmax2(as(q[i].z), as(q[i].w)));
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&top);
        return fmaxf(widen16(w & 0xFFFFu, kBf16<T>), widen16(w >> 16, kBf16<T>));
    }
}
template <typename T>
__device__ __forceinline__ uint4 narrow(const float2 (&f)[kE<T> / 2])
{
    if constexpr (sizeof(T) == 4)
        return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y),
                          __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    else
        return make_uint4(narrow32(f[0].x, f[0].y, kBf16<T>), narrow32(f[1].x, f[1].y, kBf16<T>),
                          narrow32(f[2].x, f[2].y, kBf16<T>), narrow32(f[3].x, f[3].y, kBf16<T>));
}

// A row: a head of elements up to a 16-byte boundary, whole vectors, a tail.
template <typename T>
struct Row {
    const T* p;
    int32_t head, vectors, tail;
    __device__ Row(const T* row, int32_t n) : p(row)
    {
        head = int32_t((0 - reinterpret_cast<uintptr_t>(row) / sizeof(T)) & (kE<T> - 1));
        head = head < n ? head : n;
        vectors = (n - head) / kE<T>;
        tail = n - head - vectors * kE<T>;
    }
    __device__ const uint4* body() const { return reinterpret_cast<const uint4*>(p + head); }
    // the element of the head or the tail that thread t has, or -1
    __device__ int32_t edge(int t) const
    {
        if (t < head)
            return t;
        t -= kE<T>;
        return t >= 0 && t < tail ? head + vectors * kE<T> + t : -1;
    }
};

// kAtOnce vectors of a row from v on, -inf behind its end.
template <typename T>
__device__ __forceinline__ void load_vectors(const uint4* body, int32_t v, int32_t end,
                                             uint4 (&q)[kAtOnce])
{
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
        q[i] = v + i * kThreads < end ? __ldcs(body + v + i * kThreads) : nothing<T>();
}

// (maximum, sum of 2^(x - maximum)) over a warp.
__device__ __forceinline__ void join_warp(float& most, float& sum)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float m = __shfl_xor_sync(0xFFFFFFFFu, most, off);
        const float s = __shfl_xor_sync(0xFFFFFFFFu, sum, off);
        const float now = fmaxf(most, m), base = reference(now);
        sum = sum * exp2f(most - base) + s * exp2f(m - base);
        most = now;
    }
}
__device__ __forceinline__ void join_value(float x, float& most, float& sum)
{
    const float now = fmaxf(most, x), base = reference(now);
    sum = sum * exp2f(most - base) + exp2f(x - base);
    most = now;
}

// An entry of the teacher's row: its id (-1: none, -2: past the vocabulary) and
// its value in powers of two, -inf where there is none.  A value of -inf is none
// also past the vocabulary, where a wider teacher has its masked words.
struct Entry {
    int32_t id;
    float v;
};
__device__ __forceinline__ Entry entry_of(const Distill& a, int64_t row, int32_t j, float unit)
{
    if (j >= a.k)
        return Entry{-1, -INFINITY};
    const int64_t id = a.ids[row * a.k + j];
    const float v = load_as(a.values, row * a.k + j, a.values_dtype) * unit;
    if (id < 0)
        return Entry{-1, -INFINITY};
    return Entry{id < a.vocab ? int32_t(id) : v == -INFINITY ? -1 : -2, v};
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 5) k_distill_forward(const Distill a)
{
    using namespace packed;
    __shared__ float2 slots[kWarps];
    wait_before();
    go_ahead();
    const int64_t r = blockIdx.x;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const T* const logits = static_cast<const T*>(a.logits) + r * a.stride;
    const float unit = kLog2E / a.temperature;
    const Row<T> row(logits, a.vocab);
    const uint4* const body = row.body();
    // the first warp has the teacher's entries, 32 at a time; the first of them
    // are on their way beside the row
    Entry first{-1, -INFINITY};
    if (warp == 0)
        first = entry_of(a, r, lane, unit);
    uint4 q[kAtOnce];
    load_vectors<T>(body, threadIdx.x, row.vectors, q);
    const float first_at = first.id >= 0 ? one(logits + first.id) : 0.0f;
    const int32_t edge = row.edge(threadIdx.x);
    const float edge_value = edge >= 0 ? one(logits + edge) : -INFINITY;

    float most = -INFINITY, sum = 0.0f;  // of l unit
    for (int32_t v = threadIdx.x; v < row.vectors; v += kAtOnce * kThreads) {
        const float now = fmaxf(most, largest<T>(q) * unit), base = reference(now);
        float2 add = make_float2(sum * exp2_fast(most - base), 0.0f);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
            for (int j = 0; j < kE<T> / 2; ++j)
                add = add2(add, exp2_fast(fma2(pair_of<T>(w, j), both(unit), both(-base))));
        }
        sum = add.x + add.y;
        most = now;
        load_vectors<T>(body, v + kAtOnce * kThreads, row.vectors, q);
    }
    if (edge >= 0)
        join_value(edge_value * unit, most, sum);
    join_warp(most, sum);
    if (lane == 0)
        slots[warp] = make_float2(most, sum);
    __syncthreads();
    if (warp > 0)
        return;
    const float2 mine = lane < kWarps ? slots[lane] : make_float2(-INFINITY, 0.0f);
    most = mine.x;
    sum = mine.y;
    join_warp(most, sum);
    const float lse2 = reference(most) + log2f(sum);

    float top = first.v, total = first.v == -INFINITY ? 0.0f : 1.0f;
    if (first.v != first.v)  // NaN
        top = -INFINITY, total = first.v;
    bool past = first.id == -2;
    for (int32_t j = 32 + lane; j < a.k; j += 32) {
        const Entry e = entry_of(a, r, j, unit);
        past |= e.id == -2;
        join_value(e.v, top, total);
    }
    join_warp(top, total);
    past = __any_sync(0xFFFFFFFFu, past);
    float loss = 0.0f;
    if (total != 0.0f) {
        const float base = reference(top), log_total = log2f(total);
        for (int32_t j = lane; j < a.k; j += 32) {
            const Entry e = j == lane ? first : entry_of(a, r, j, unit);
            const float log_q = e.v - base - log_total, p = exp2f(log_q);
            if (p != 0.0f && e.id >= 0)
                loss += p * (log_q - ((j == lane ? first_at : one(logits + e.id)) * unit - lse2));
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        loss += __shfl_xor_sync(0xFFFFFFFFu, loss, off);
    if (lane == 0) {
        a.loss[r] = past ? NAN : loss * (a.temperature * a.temperature * kLn2);
        if (a.lse)
            a.lse[r] = lse2 * kLn2;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 4 : 5)
    k_distill_backward(const Distill a)
{
    using namespace packed;
    __shared__ int32_t ids[kDistillMost];
    __shared__ float values[kDistillMost], at[kDistillMost];
    __shared__ float2 teacher;
    __shared__ bool id_past;
    wait_before();
    go_ahead();
    const int64_t r = blockIdx.x;
    const int lane = threadIdx.x % 32;
    const T* const logits = static_cast<const T*>(a.logits) + r * a.stride;
    T* const out = static_cast<T*>(a.dlogits) + r * a.dlogits_stride;
    const float unit = kLog2E / a.temperature;
    const Row<T> row(logits, a.vocab);
    const uint4* const body = row.body();
    uint4 q[kAtOnce];
    load_vectors<T>(body, threadIdx.x, row.vectors, q);
    const int32_t edge = row.edge(threadIdx.x);
    const float edge_value = edge >= 0 ? one(logits + edge) : 0.0f;
    const float factor = a.temperature * a.scale * (a.dloss ? a.dloss[r] : 1.0f);
    const float base = a.lse_in[r] * kLog2E;
    // the first warp reads the teacher's entries, and the logits there before
    // anything is written: out may be the logits
    if (threadIdx.x < 32) {
        float top = -INFINITY, total = 0.0f;
        bool past = false;
        for (int32_t j = lane; j < a.k; j += 32) {
            const Entry e = entry_of(a, r, j, unit);
            past |= e.id == -2;
            ids[j] = e.id;
            values[j] = e.v;
            at[j] = e.id >= 0 ? one(logits + e.id) : 0.0f;
            join_value(e.v, top, total);
        }
        join_warp(top, total);
        past = __any_sync(0xFFFFFFFFu, past);
        if (lane == 0) {
            teacher = make_float2(reference(top), total);
            id_past = past;
        }
    }
    __syncthreads();
    const bool past = id_past, some = teacher.y != 0.0f;
    // T scale (p): p times factor, or what a row without entries or with a bad
    // one gets instead
    const float flat = past ? NAN : 0.0f;
    const bool is_flat = past || !some;
    const auto gradient = [&](float2 l) {
        const float2 g = mul2(exp2_fast(fma2(l, both(unit), both(-base))), both(factor));
        return is_flat ? both(flat) : g;
    };
    if ((reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(out)) % 16 == 0) {
        uint4* const to = reinterpret_cast<uint4*>(out + row.head);
        for (int32_t v = threadIdx.x; v < row.vectors; v += kAtOnce * kThreads) {
            uint4 next[kAtOnce];
            load_vectors<T>(body, v + kAtOnce * kThreads, row.vectors, next);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
                float2 f[kE<T> / 2];
#pragma unroll
                for (int j = 0; j < kE<T> / 2; ++j)
                    f[j] = gradient(pair_of<T>(w, j));
                if (v + i * kThreads < row.vectors)
                    to[v + i * kThreads] = narrow<T>(f);
                q[i] = next[i];
            }
        }
        if (edge >= 0)
            put(out + edge, gradient(make_float2(edge_value, 0.0f)).x);
    } else {
#pragma unroll 8
        for (int32_t c = threadIdx.x; c < a.vocab; c += kThreads)
            put(out + c, gradient(make_float2(one(logits + c), 0.0f)).x);
    }
    if (is_flat)
        return;
    // the teacher's probabilities, at the k places; an id that is there twice
    // gets the sum both times
    const float inverse = 1.0f / teacher.y;
    for (int32_t j = threadIdx.x; j < a.k; j += kThreads)
        values[j] = exp2f(values[j] - teacher.x) * inverse;
    __syncthreads();
    for (int32_t j = threadIdx.x; j < a.k; j += kThreads) {
        const int32_t id = ids[j];
        if (id < 0)
            continue;
        float p = 0.0f;
        for (int32_t i = 0; i < a.k; ++i)
            p += ids[i] == id ? values[i] : 0.0f;
        put(out + id, (exp2f(fmaf(at[j], unit, -base)) - p) * factor);
    }
}

template <typename F>
int by_type(int32_t dtype, F&& f)
{
    switch (dtype) {
    case ADAMW_DTYPE_F32: return f(float());
    case ADAMW_DTYPE_BF16: return f(__nv_bfloat16());
    default: return f(__half());
    }
}

}  // namespace

int launch_distill_forward(const Distill& a, void* stream)
{
    return by_type(a.dtype, [&](auto t) {
        return launch_early(k_distill_forward<decltype(t)>, dim3(unsigned(a.rows)), kThreads, 0,
                            static_cast<cudaStream_t>(stream), a);
    });
}
int launch_distill_backward(const Distill& a, void* stream)
{
    return by_type(a.dtype, [&](auto t) {
        return launch_early(k_distill_backward<decltype(t)>, dim3(unsigned(a.rows)), kThreads, 0,
                            static_cast<cudaStream_t>(stream), a);
    });
}

}  // namespace osr
