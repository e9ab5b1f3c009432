// layernorm_bwd.cuh -- the layer norm's backward pass, for sm_103a; one
// translation unit per element type instantiates it.
//
// "Grow a Language Model: Backprop" (unhomeschool.com), section "Every
// forward op gets a backward twin": each backward kernel computes the
// gradient of its input and of its weights in one launch.  With xhat = (x -
// mean) rstd and a = dy w:
//   dx = rstd (a - mean(a) - xhat mean(a xhat))
//   dweight = sum over rows of dy xhat,  dbias = sum over rows of dy.
// HBM-bound: x and dy are read once and dx is written once.  A thread owns
// the same columns in every row it sees, so the two column sums stay in its
// registers until the end; each block then writes its share (2 cols floats),
// and k_ln_grads (layernorm_bwd.cu) joins the blocks' shares in a fixed order.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "layernorm_dev.cuh"

namespace osr {
namespace {

using namespace ln;

// Resident blocks the kernel is compiled for: 16 kVecs registers hold a
// thread's column sums, 8 kVecs its weights.
template <int kGroup, int kVecs>
constexpr int kBackwardBlocks = (kVecs == 1 ? 768 : kVecs == 2 ? 640 : 512) / kBlockThreads<kGroup>;

template <typename T, int kGroup, int kVecs>
using BackwardRing =
    Ring<T, kBlockThreads<kGroup>, kVecs, 2,
         stages_for(2 * kVecs * kBlockThreads<kGroup> * kE * int(sizeof(T)),
                    kBackwardBlocks<kGroup, kVecs>)>;

// A row is looked at twice in shared memory, for the sums and for dx, rather
// than kept widened in 16 kVecs more registers.
template <typename T, int kGroup, int kVecs, bool kRagged>
__global__ void __launch_bounds__(kBlockThreads<kGroup>, (kBackwardBlocks<kGroup, kVecs>))
    k_ln_backward(LnBackward a)
{
    constexpr int kThreads = kBlockThreads<kGroup>;
    constexpr int kGroups = kThreads / kGroup;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(16) unsigned char raw[];
    const BackwardRing<T, kGroup, kVecs> ring{reinterpret_cast<uint4*>(raw)};
    constexpr int kStages = BackwardRing<T, kGroup, kVecs>::kDepth;
    __shared__ float2 slots[2][32];
    int turn = 0;
    const int lane = threadIdx.x % kGroup;
    const int64_t group = int64_t(blockIdx.x) * kGroups + threadIdx.x / kGroup;
    const int64_t groups = int64_t(gridDim.x) * kGroups;
    const T* const x = static_cast<const T*>(a.x);
    const T* const dy = static_cast<const T*>(a.dy);
    T* const dx = static_cast<T*>(a.dx);
    const int cols = a.cols;
    const int off = kRagged ? offset_of(x + group * a.x_stride) : 0;
    const bool dy_whole = !kRagged || offset_of(dy + group * a.dy_stride) == off;
    const bool dx_whole = !kRagged || offset_of(dx + group * a.dx_stride) == off;
    auto column = [&](int v) { return (v * kGroup + lane) * kE - off; };
    float next_mean[kStages], next_rstd[kStages];  // [i]: of the row i + 1 turns ahead
    auto fetch = [&](int stage, int64_t r, float& mean, float& rstd) {
        const bool live = r < a.rows;
        if (live) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const int c = column(v);
                if (is_full<kRagged>(c, cols)) {
                    ring.copy(stage, 0, v, x + r * a.x_stride + c);
                    if (dy_whole)
                        ring.copy(stage, 1, v, dy + r * a.dy_stride + c);
                }
            }
        }
        mean = live ? a.mean[r] : 0.0f;
        rstd = live ? a.rstd[r] : 0.0f;
        commit_copies();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        fetch(i, group + i * groups, next_mean[i], next_rstd[i]);

    float w[kVecs][kE], dw[kVecs][kE], db[kVecs][kE];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        load_weight<T>(a.weight, a.w_f32, column(v), cols, 1.0f, w[v]);
#pragma unroll
        for (int i = 0; i < kE; ++i)
            dw[v][i] = db[v][i] = 0.0f;
    }
    const float inv = 1.0f / float(cols);
    int stage = 0;
    for (int64_t first = group - threadIdx.x / kGroup; first < a.rows; first += groups) {
        const int64_t r = first + threadIdx.x / kGroup;
        const bool live = r < a.rows;
        fetch(stage == 0 ? kStages - 1 : stage - 1, r + (kStages - 1) * groups,
              next_mean[kStages - 1], next_rstd[kStages - 1]);
        const float mean = next_mean[0], rstd = next_rstd[0];
#pragma unroll
        for (int i = 0; i + 1 < kStages; ++i) {
            next_mean[i] = next_mean[i + 1];
            next_rstd[i] = next_rstd[i + 1];
        }
        wait_copies<kStages - 1>();
        // one vector of the row, as xhat and dy; outside the row dy is 0, and
        // so are all sums
        auto take = [&](int v, float(&xh)[kE], float(&g)[kE]) {
            const int c = column(v);
            const bool full = live && is_full<kRagged>(c, cols);
            if (full) {
                ring.read(stage, 0, v, xh);
            } else if (kRagged && live) {
                load_elements(x + r * a.x_stride, c, cols, xh);
            } else {
#pragma unroll
                for (int i = 0; i < kE; ++i)
                    xh[i] = 0.0f;
            }
            if (full && dy_whole) {
                ring.read(stage, 1, v, g);
            } else if (kRagged && live) {
                load_elements(dy + r * a.dy_stride, c, cols, g);
            } else {
#pragma unroll
                for (int i = 0; i < kE; ++i)
                    g[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < kE; ++i)
                xh[i] = (xh[i] - mean) * rstd;
        };
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            float xh[kE], g[kE];
            take(v, xh, g);
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                dw[v][i] += g[i] * xh[i];
                db[v][i] += g[i];
                g[i] *= w[v][i];
                s1 += g[i];
                s2 += g[i] * xh[i];
            }
        }
        const float2 s = group_sum<kGroup>(s1, s2, slots, turn);
        const float m1 = s.x * inv, m2 = s.y * inv;
        if (live) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                float xh[kE], g[kE];
                take(v, xh, g);
#pragma unroll
                for (int i = 0; i < kE; ++i)
                    g[i] = rstd * (g[i] * w[v][i] - m1 - xh[i] * m2);
                store_vec<kRagged>(dx + r * a.dx_stride, column(v), cols, dx_whole, g);
            }
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    wait_copies<0>();
    if (!a.sums)
        return;

    float* const mine = a.partials + int64_t(blockIdx.x) * 2 * cols;
    if constexpr (kGroups == 1) {
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                const int c = column(v) + i;
                if (c >= 0 && c < cols) {
                    mine[c] = dw[v][i];
                    mine[cols + c] = db[v][i];
                }
            }
    } else {
        // the block's groups join by columns (their offsets may differ), in
        // the memory of the ring
        constexpr int kSpan = kGroup * kVecs * kE;
        float* const part = reinterpret_cast<float*>(raw);
        static_assert(kGroups * kSpan * 4 <= BackwardRing<T, kGroup, kVecs>::kBytes,
                      "the sums fit the ring");
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
#pragma unroll
                for (int i = 0; i < kE; ++i) {
                    const int c = column(v) + i;
                    if (c >= 0 && c < cols)
                        part[threadIdx.x / kGroup * kSpan + c] = pass ? db[v][i] : dw[v][i];
                }
            __syncthreads();
            for (int c = threadIdx.x; c < cols; c += kThreads) {
                float s = 0.0f;
#pragma unroll
                for (int q = 0; q < kGroups; ++q)
                    s += part[q * kSpan + c];
                mine[pass * cols + c] = s;
            }
        }
    }
}

// Rows that do not fit a block's registers.  dx: two looks at each row, the
// second from L2.
constexpr int kWideThreads = 512;

template <typename T>
__device__ __forceinline__ float weight_at(const LnBackward& a, int c)
{
    return !a.weight ? 1.0f
           : a.w_f32 ? static_cast<const float*>(a.weight)[c]
                     : detail::load1(static_cast<const T*>(a.weight) + c);
}

template <typename T>
__global__ void __launch_bounds__(kWideThreads) k_ln_backward_wide(LnBackward a)
{
    __shared__ float2 slots[2][32];
    int turn = 0;
    const int cols = a.cols;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* const x = static_cast<const T*>(a.x) + r * a.x_stride;
        const T* const dy = static_cast<const T*>(a.dy) + r * a.dy_stride;
        T* const dx = static_cast<T*>(a.dx) + r * a.dx_stride;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x; c < cols; c += kWideThreads) {
            const float g = detail::load1(dy + c) * weight_at<T>(a, c);
            s1 += g;
            s2 += g * (detail::load1(x + c) - mean) * rstd;
        }
        const float2 s = group_sum<kWideThreads>(s1, s2, slots, turn);
        const float m1 = s.x / float(cols), m2 = s.y / float(cols);
        for (int c = threadIdx.x; c < cols; c += kWideThreads) {
            const float g = detail::load1(dy + c) * weight_at<T>(a, c);
            store_one(dx + c, rstd * (g - m1 - (detail::load1(x + c) - mean) * rstd * m2));
        }
    }
}

// The column sums of such rows: a thread per column, a strip of rows per
// block of the grid's second dimension.
template <typename T>
__global__ void __launch_bounds__(256) k_ln_columns_wide(LnBackward a)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.cols)
        return;
    const int64_t lo = a.rows * blockIdx.y / gridDim.y, hi = a.rows * (blockIdx.y + 1) / gridDim.y;
    const T* x = static_cast<const T*>(a.x) + lo * a.x_stride + c;
    const T* dy = static_cast<const T*>(a.dy) + lo * a.dy_stride + c;
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = lo; r < hi; ++r, x += a.x_stride, dy += a.dy_stride) {
        const float g = detail::load1(dy);
        dw += g * (detail::load1(x) - a.mean[r]) * a.rstd[r];
        db += g;
    }
    float* const mine = a.partials + int64_t(blockIdx.y) * 2 * a.cols;
    mine[c] = dw;
    mine[a.cols + c] = db;
}

template <typename T, int G, int V, bool kRagged>
int launch_one(const LnBackward& a, int sm_count, int32_t* parts, cudaStream_t s)
{
    constexpr int kThreads = kBlockThreads<G>;
    constexpr int kSmem = BackwardRing<T, G, V>::kBytes;
    auto* const kernel = &k_ln_backward<T, G, V, kRagged>;
    static const int cap = resident_blocks(kernel, kThreads, kSmem);
    int64_t blocks = detail::ceil_div(a.rows, kThreads / G);
    if (kThreads / G < kE)
        blocks = detail::ceil_div(blocks, kE) * kE;  // groups step by a multiple of 8
    int64_t most = int64_t(cap) * sm_count;
    if (most > ln_parts_max(a.cols))
        most = ln_parts_max(a.cols);
    most = most / kE * kE;
    blocks = blocks > most ? most : blocks;
    *parts = int32_t(blocks);
    kernel<<<unsigned(blocks), kThreads, kSmem, s>>>(a);
    return int(cudaGetLastError());
}

}  // namespace

template <typename T>
int launch_ln_backward_typed(const LnBackward& a, int sm_count, int32_t* parts, cudaStream_t s)
{
    const bool aligned = a.cols % kE == 0 && rows_aligned<T>(a.x, a.x_stride) &&
                         rows_aligned<T>(a.dy, a.dy_stride) && rows_aligned<T>(a.dx, a.dx_stride);
    const int span = aligned ? a.cols : a.cols + kE - 1;
    if (span > kLnRegisterCols) {
        const int64_t most = int64_t(sm_count) * 4;
        k_ln_backward_wide<T>
            <<<unsigned(a.rows < most ? a.rows : most), kWideThreads, 0, s>>>(a);
        const cudaError_t e = cudaGetLastError();
        *parts = int32_t(a.rows < kLnWideParts ? a.rows : kLnWideParts);
        if (e != cudaSuccess || !a.sums)
            return int(e);
        k_ln_columns_wide<T>
            <<<dim3(unsigned(detail::ceil_div(a.cols, 256)), unsigned(*parts)), 256, 0, s>>>(a);
        return int(cudaGetLastError());
    }
    return with_layout(span, [&](auto layout) {
        constexpr int G = decltype(layout)::kGroup, V = decltype(layout)::kVecs;
        return aligned ? launch_one<T, G, V, false>(a, sm_count, parts, s)
                       : launch_one<T, G, V, true>(a, sm_count, parts, s);
    });
}

}  // namespace osr
