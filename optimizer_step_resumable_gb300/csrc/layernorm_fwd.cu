// layernorm_fwd.cu -- the layer norm's forward pass, for sm_103a.
//
// "Grow a Language Model: Backprop" (unhomeschool.com), section "Every
// forward op gets a backward twin": k_layernorm_fwd keeps each row's mean and
// variance for the backward pass.  HBM-bound: every element is read once and
// written once; the mean and then the squares of the differences are summed
// from registers, so the variance loses nothing to cancellation.
#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "layernorm_dev.cuh"

namespace osr {
namespace {

using namespace ln;

// Resident blocks the kernel is compiled for: 24 kVecs registers hold a
// thread's weights, biases and elements.
template <int kGroup, int kVecs>
constexpr int kForwardBlocks = (kVecs == 1 ? 1024 : 512) / kBlockThreads<kGroup>;

template <typename T, int kGroup, int kVecs>
using ForwardRing =
    Ring<T, kBlockThreads<kGroup>, kVecs, 1,
         stages_for(kVecs * kBlockThreads<kGroup> * kE * int(sizeof(T)),
                    kForwardBlocks<kGroup, kVecs>)>;

template <typename T, int kGroup, int kVecs, bool kRagged>
__global__ void __launch_bounds__(kBlockThreads<kGroup>, (kForwardBlocks<kGroup, kVecs>))
    k_ln_forward(LnForward a)
{
    constexpr int kThreads = kBlockThreads<kGroup>;
    constexpr int kGroups = kThreads / kGroup;
    extern __shared__ __align__(16) unsigned char raw[];
    const ForwardRing<T, kGroup, kVecs> ring{reinterpret_cast<uint4*>(raw)};
    constexpr int kStages = ForwardRing<T, kGroup, kVecs>::kDepth;
    __shared__ float2 slots[2][32];
    int turn = 0;
    const int lane = threadIdx.x % kGroup;
    const int64_t group = int64_t(blockIdx.x) * kGroups + threadIdx.x / kGroup;
    const int64_t groups = int64_t(gridDim.x) * kGroups;
    const T* const x = static_cast<const T*>(a.x);
    T* const y = static_cast<T*>(a.y);
    const int cols = a.cols;
    const int off = kRagged ? offset_of(x + group * a.x_stride) : 0;
    const bool y_whole = !kRagged || offset_of(y + group * a.y_stride) == off;
    auto column = [&](int v) { return (v * kGroup + lane) * kE - off; };
    auto fetch = [&](int stage, int64_t r) {
        if (r < a.rows) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
                if (is_full<kRagged>(column(v), cols))
                    ring.copy(stage, 0, v, x + r * a.x_stride + column(v));
        }
        commit_copies();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        fetch(i, group + i * groups);

    float w[kVecs][kE], b[kVecs][kE];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        load_weight<T>(a.weight, a.w_f32, column(v), cols, 1.0f, w[v]);
        load_weight<T>(a.bias, a.w_f32, column(v), cols, 0.0f, b[v]);
    }
    // every thread takes part in every sum: the rows past the end are empty
    const float inv = 1.0f / float(cols);
    int stage = 0;
    for (int64_t first = group - threadIdx.x / kGroup; first < a.rows; first += groups) {
        const int64_t r = first + threadIdx.x / kGroup;
        const bool live = r < a.rows;
        fetch(stage == 0 ? kStages - 1 : stage - 1, r + (kStages - 1) * groups);
        wait_copies<kStages - 1>();
        float f[kVecs][kE];
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int c = column(v);
            if (live && is_full<kRagged>(c, cols)) {
                ring.read(stage, 0, v, f[v]);
            } else if (kRagged && live) {
                load_elements(x + r * a.x_stride, c, cols, f[v]);
            } else {
#pragma unroll
                for (int i = 0; i < kE; ++i)
                    f[v][i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < kE; ++i)
                sum += f[v][i];
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
        const float mean = group_sum<kGroup>(sum, 0.0f, slots, turn).x * inv;
        float squares = 0.0f;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int c = column(v);
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                f[v][i] -= mean;
                if (in_row<kRagged>(c, i, cols))
                    squares += f[v][i] * f[v][i];
            }
        }
        const float var = group_sum<kGroup>(squares, 0.0f, slots, turn).x * inv;
        const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(var + a.eps));
        if (!live)
            continue;
        T* const yr = y + r * a.y_stride;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            float o[kE];
#pragma unroll
            for (int i = 0; i < kE; ++i)
                o[i] = f[v][i] * rstd * w[v][i] + b[v][i];
            store_vec<kRagged>(yr, column(v), cols, y_whole, o);
        }
        if (lane == 0) {
            if (a.mean)
                a.mean[r] = mean;
            if (a.rstd)
                a.rstd[r] = rstd;
        }
    }
}

// Rows that do not fit a block's registers: three looks at the row, the
// later two from L2 or L1.
constexpr int kWideThreads = 512;

template <typename T>
__global__ void __launch_bounds__(kWideThreads) k_ln_forward_wide(LnForward a)
{
    __shared__ float2 slots[2][32];
    int turn = 0;
    const int cols = a.cols;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* const x = static_cast<const T*>(a.x) + r * a.x_stride;
        T* const y = static_cast<T*>(a.y) + r * a.y_stride;
        float sum = 0.0f;
        for (int c = threadIdx.x; c < cols; c += kWideThreads)
            sum += detail::load1(x + c);
        const float mean = group_sum<kWideThreads>(sum, 0.0f, slots, turn).x / float(cols);
        float squares = 0.0f;
        for (int c = threadIdx.x; c < cols; c += kWideThreads) {
            const float d = detail::load1(x + c) - mean;
            squares += d * d;
        }
        const float var = group_sum<kWideThreads>(squares, 0.0f, slots, turn).x / float(cols);
        const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(var + a.eps));
        for (int c = threadIdx.x; c < cols; c += kWideThreads) {
            const float w = !a.weight ? 1.0f
                            : a.w_f32 ? static_cast<const float*>(a.weight)[c]
                                      : detail::load1(static_cast<const T*>(a.weight) + c);
            const float b = !a.bias  ? 0.0f
                            : a.w_f32 ? static_cast<const float*>(a.bias)[c]
                                      : detail::load1(static_cast<const T*>(a.bias) + c);
            store_one(y + c, (detail::load1(x + c) - mean) * rstd * w + b);
        }
        if (threadIdx.x == 0) {
            if (a.mean)
                a.mean[r] = mean;
            if (a.rstd)
                a.rstd[r] = rstd;
        }
    }
}

template <typename T, int G, int V, bool kRagged>
int launch_one(const LnForward& a, int sm_count, cudaStream_t s)
{
    constexpr int kThreads = kBlockThreads<G>;
    constexpr int kSmem = ForwardRing<T, G, V>::kBytes;
    auto* const kernel = &k_ln_forward<T, G, V, kRagged>;
    static const int cap = resident_blocks(kernel, kThreads, kSmem);
    int64_t blocks = detail::ceil_div(a.rows, kThreads / G);
    if (kThreads / G < kE)
        blocks = detail::ceil_div(blocks, kE) * kE;  // groups step by a multiple of 8
    const int64_t most = int64_t(cap) * sm_count / kE * kE;
    blocks = blocks > most ? most : blocks;
    kernel<<<unsigned(blocks), kThreads, kSmem, s>>>(a);
    return int(cudaGetLastError());
}

template <typename T>
int launch_typed(const LnForward& a, int sm_count, cudaStream_t s)
{
    const bool aligned = a.cols % kE == 0 && rows_aligned<T>(a.x, a.x_stride) &&
                         rows_aligned<T>(a.y, a.y_stride);
    const int span = aligned ? a.cols : a.cols + kE - 1;
    if (span > kLnRegisterCols) {
        const int64_t most = int64_t(sm_count) * 4;
        k_ln_forward_wide<T><<<unsigned(a.rows < most ? a.rows : most), kWideThreads, 0, s>>>(a);
        return int(cudaGetLastError());
    }
    return with_layout(span, [&](auto layout) {
        constexpr int G = decltype(layout)::kGroup, V = decltype(layout)::kVecs;
        return aligned ? launch_one<T, G, V, false>(a, sm_count, s)
                       : launch_one<T, G, V, true>(a, sm_count, s);
    });
}

}  // namespace

int launch_ln_forward(const LnForward& a, int32_t dtype, int sm_count, void* stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == kDtypeBF16)
        return launch_typed<__nv_bfloat16>(a, sm_count, s);
    if (dtype == kDtypeF16)
        return launch_typed<__half>(a, sm_count, s);
    return launch_typed<float>(a, sm_count, s);
}

}  // namespace osr
