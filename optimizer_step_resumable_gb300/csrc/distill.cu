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

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr float kLn2 = 0.69314718055994531f;

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
template <typename T>
__device__ __forceinline__ void widen(uint4 q, float (&f)[kE<T>])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if constexpr (sizeof(T) == 4) {
            f[i] = __uint_as_float(w[i]);
        } else {
            f[2 * i] = widen16(w[i] & 0xFFFFu, kBf16<T>);
            f[2 * i + 1] =
                kBf16<T> ? __uint_as_float(w[i] & 0xFFFF0000u) : widen16(w[i] >> 16, false);
        }
}
template <typename T>
__device__ __forceinline__ uint4 narrow(const float (&f)[kE<T>])
{
    if constexpr (sizeof(T) == 4)
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    else
        return make_uint4(narrow32(f[0], f[1], kBf16<T>), narrow32(f[2], f[3], kBf16<T>),
                          narrow32(f[4], f[5], kBf16<T>), narrow32(f[6], f[7], kBf16<T>));
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

// (maximum, sum of 2^(x - maximum)) over the block, in every thread.
__device__ float2 join_block(float most, float sum, float2 (&slots)[kWarps])
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float m = __shfl_xor_sync(0xFFFFFFFFu, most, off);
        const float s = __shfl_xor_sync(0xFFFFFFFFu, sum, off);
        const float now = fmaxf(most, m), base = reference(now);
        sum = sum * exp2f(most - base) + s * exp2f(m - base);
        most = now;
    }
    __syncthreads();  // the slots of the call before
    if (threadIdx.x % 32 == 0)
        slots[threadIdx.x / 32] = make_float2(most, sum);
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        top = fmaxf(top, slots[w].x);
    const float base = reference(top);
    float total = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        total += slots[w].y * exp2f(slots[w].x - base);
    return make_float2(top, total);
}

// The teacher's row: ids, values in powers of two, the row's logits there,
// and whether an id is past the vocabulary.
struct Teacher {
    int32_t id[kDistillMost];
    float q[kDistillMost];
    float at[kDistillMost];
    int32_t past;
};
// Whether there is an entry at all; total: their maximum and sum.
template <typename T>
__device__ __forceinline__ bool read_teacher(const Distill& a, int64_t row, const T* logits,
                                             Teacher& t, float2 (&slots)[kWarps], float2& total)
{
    const float unit = kLog2E / a.temperature;
    if (threadIdx.x == 0)
        t.past = 0;
    __syncthreads();
    float most = -INFINITY;
    for (int32_t j = threadIdx.x; j < a.k; j += kThreads) {
        const int64_t id = a.ids[row * a.k + j];
        const bool there = id >= 0 && id < a.vocab;
        if (id >= a.vocab)
            t.past = 1;
        const float v = id >= 0 ? load_as(a.values, row * a.k + j, a.values_dtype) * unit
                                : -INFINITY;
        t.id[j] = there ? int32_t(id) : -1;
        t.q[j] = v;
        t.at[j] = there ? one(logits + id) : 0.0f;
        most = fmaxf(most, v);
    }
    float sum = 0.0f;
    const float base = reference(most);
    for (int32_t j = threadIdx.x; j < a.k; j += kThreads)
        sum += exp2f(t.q[j] - base);
    total = join_block(most, sum, slots);
    return total.y != 0.0f;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) k_distill_forward(const Distill a)
{
    __shared__ Teacher t;
    __shared__ float2 slots[kWarps];
    __shared__ float sums[kWarps];
    wait_before();
    go_ahead();
    const int64_t r = blockIdx.x;
    const T* const logits = static_cast<const T*>(a.logits) + r * a.stride;
    const float unit = kLog2E / a.temperature;
    float most = -INFINITY, sum = 0.0f;  // of l unit
    const Row<T> row(logits, a.vocab);
    const uint4* const body = row.body();
    constexpr int kAtOnce = 4, kMany = kAtOnce * kE<T>;
    for (int32_t v = threadIdx.x; v < row.vectors; v += kAtOnce * kThreads) {
        float f[kMany];
        uint4 q[kAtOnce] = {};
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (v + i * kThreads < row.vectors)
                q[i] = __ldcs(body + v + i * kThreads);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            float g[kE<T>];
            widen<T>(q[i], g);
#pragma unroll
            for (int j = 0; j < kE<T>; ++j)
                f[i * kE<T> + j] = v + i * kThreads < row.vectors ? g[j] : -INFINITY;
        }
        float top = f[0];
#pragma unroll
        for (int j = 1; j < kMany; ++j)
            top = fmaxf(top, f[j]);
        const float now = fmaxf(most, top * unit), base = reference(now);
        sum *= exp2_fast(most - base);
        float add[4] = {};
#pragma unroll
        for (int j = 0; j < kMany; ++j)
            add[j % 4] += exp2_fast(fmaf(f[j], unit, -base));
        sum += (add[0] + add[1]) + (add[2] + add[3]);
        most = now;
    }
    const int32_t edge = row.edge(threadIdx.x);
    if (edge >= 0) {
        const float x = one(logits + edge) * unit, now = fmaxf(most, x), base = reference(now);
        sum = sum * exp2_fast(most - base) + exp2_fast(x - base);
        most = now;
    }
    const float2 all = join_block(most, sum, slots);
    const float lse2 = reference(all.x) + log2f(all.y);
    float2 total;
    const bool some = read_teacher(a, r, logits, t, slots, total);
    const float base = reference(total.x), log_total = log2f(total.y);
    float loss = 0.0f;
    if (some)
        for (int32_t j = threadIdx.x; j < a.k; j += kThreads) {
            const float log_q = t.q[j] - base - log_total, q = exp2f(log_q);
            if (q != 0.0f)
                loss += q * (log_q - (t.at[j] * unit - lse2));
        }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        loss += __shfl_xor_sync(0xFFFFFFFFu, loss, off);
    if (threadIdx.x % 32 == 0)
        sums[threadIdx.x / 32] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
        loss = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            loss += sums[w];
        loss *= a.temperature * a.temperature * kLn2;
        a.loss[r] = t.past ? NAN : loss;
        if (a.lse)
            a.lse[r] = lse2 * kLn2;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) k_distill_backward(const Distill a)
{
    __shared__ Teacher t;
    __shared__ float2 slots[kWarps];
    wait_before();
    go_ahead();
    const int64_t r = blockIdx.x;
    const T* const logits = static_cast<const T*>(a.logits) + r * a.stride;
    T* const out = static_cast<T*>(a.dlogits) + r * a.dlogits_stride;
    const float unit = kLog2E / a.temperature;
    float2 total;
    // before anything is written: out may be the logits
    const bool some = read_teacher(a, r, logits, t, slots, total);
    const float factor = a.temperature * a.scale * (a.dloss ? a.dloss[r] : 1.0f);
    const float base = a.lse_in[r] * kLog2E;
    const bool past = t.past;
    const auto gradient = [&](float l) {
        const float g = exp2_fast(fmaf(l, unit, -base)) * factor;
        return past ? NAN : some ? g : 0.0f;
    };
    const Row<T> row(logits, a.vocab);
    const uint4* const body = row.body();
    if ((reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(out)) % 16 == 0) {
        uint4* const to = reinterpret_cast<uint4*>(out + row.head);
        constexpr int kAtOnce = 4;
        for (int32_t v = threadIdx.x; v < row.vectors; v += kAtOnce * kThreads) {
            uint4 q[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (v + i * kThreads < row.vectors)
                    q[i] = __ldcs(body + v + i * kThreads);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (v + i * kThreads < row.vectors) {
                    float f[kE<T>];
                    widen<T>(q[i], f);
#pragma unroll
                    for (int j = 0; j < kE<T>; ++j)
                        f[j] = gradient(f[j]);
                    to[v + i * kThreads] = narrow<T>(f);
                }
        }
        const int32_t edge = row.edge(threadIdx.x);
        if (edge >= 0)
            put(out + edge, gradient(one(logits + edge)));
    } else {
#pragma unroll 8
        for (int32_t c = threadIdx.x; c < a.vocab; c += kThreads)
            put(out + c, gradient(one(logits + c)));
    }
    if (!some || past)
        return;
    // the teacher's probabilities, at the k places; an id that is there twice
    // gets the sum both times
    const float top = reference(total.x), inverse = 1.0f / total.y;
    for (int32_t j = threadIdx.x; j < a.k; j += kThreads)
        t.q[j] = exp2f(t.q[j] - top) * inverse;
    __syncthreads();
    for (int32_t j = threadIdx.x; j < a.k; j += kThreads) {
        const int32_t id = t.id[j];
        if (id < 0)
            continue;
        float q = 0.0f;
        for (int32_t i = 0; i < a.k; ++i)
            q += t.id[i] == id ? t.q[i] : 0.0f;
        put(out + id, (exp2f(fmaf(t.at[j], unit, -base)) - q) * factor);
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
