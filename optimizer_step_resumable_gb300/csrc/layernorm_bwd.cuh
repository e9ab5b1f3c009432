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

template <typename T, int kGroup, int kVecs, bool kRagged>
__global__ void __launch_bounds__(kBlockThreads<kGroup>)
    k_ln_backward(LnBackward a)
{
    constexpr int kThreads = kBlockThreads<kGroup>;
    constexpr int kGroups = kThreads / kGroup;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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

    float w[kVecs][kE], dw[kVecs][kE], db[kVecs][kE];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        load_weight<T>(a.weight, a.w_f32, (v * kGroup + lane) * kE - off, cols, 1.0f, w[v]);
#pragma unroll
        for (int i = 0; i < kE; ++i)
            dw[v][i] = db[v][i] = 0.0f;
    }
    const float inv = 1.0f / float(cols);
    for (int64_t first = group - threadIdx.x / kGroup; first < a.rows; first += groups) {
        const int64_t r = first + threadIdx.x / kGroup;
        const bool live = r < a.rows;
        const float mean = live ? a.mean[r] : 0.0f, rstd = live ? a.rstd[r] : 0.0f;
        const int end = live ? cols : INT32_MIN;
        float xh[kVecs][kE], g[kVecs][kE];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int c = (v * kGroup + lane) * kE - off;
            load8<kRagged>(x + r * a.x_stride, c, end, true, xh[v]);
            load8<kRagged>(dy + r * a.dy_stride, c, end, dy_whole, g[v]);
        }
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int i = 0; i < kE; ++i) {  // outside the row dy is 0, and so are all sums
                xh[v][i] = (xh[v][i] - mean) * rstd;
                dw[v][i] += g[v][i] * xh[v][i];
                db[v][i] += g[v][i];
                g[v][i] *= w[v][i];
                s1 += g[v][i];
                s2 += g[v][i] * xh[v][i];
            }
        const float2 s = group_sum<kGroup>(s1, s2, slots, turn);
        if (!live)
            continue;
        const float m1 = s.x * inv, m2 = s.y * inv;
        T* const dxr = dx + r * a.dx_stride;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int c = (v * kGroup + lane) * kE - off;
            float o[kE];
#pragma unroll
            for (int i = 0; i < kE; ++i)
                o[i] = rstd * (g[v][i] - m1 - xh[v][i] * m2);
            store8<kRagged>(dxr, c, cols, dx_whole, o);
        }
    }
    if (!a.sums)
        return;

    float* const mine = a.partials + int64_t(blockIdx.x) * 2 * cols;
    if constexpr (kGroups == 1) {
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                const int c = (v * kGroup + lane) * kE - off + i;
                if (c >= 0 && c < cols) {
                    mine[c] = dw[v][i];
                    mine[cols + c] = db[v][i];
                }
            }
    } else {
        // the block's groups join by columns: their offsets may differ
        constexpr int kSpan = kGroup * kVecs * kE;
        __shared__ float part[kGroups][kSpan];
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            __syncthreads();
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
#pragma unroll
                for (int i = 0; i < kE; ++i) {
                    const int c = (v * kGroup + lane) * kE - off + i;
                    if (c >= 0 && c < cols)
                        part[threadIdx.x / kGroup][c] = pass ? db[v][i] : dw[v][i];
                }
            __syncthreads();
            for (int c = threadIdx.x; c < cols; c += kThreads) {
                float s = 0.0f;
#pragma unroll
                for (int q = 0; q < kGroups; ++q)
                    s += part[q][c];
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
    cudaError_t err = cudaSuccess;
    static const int cap = detail::resident_blocks(
        reinterpret_cast<const void*>(&k_ln_backward<T, G, V, kRagged>), kThreads, 1, &err);
    int64_t blocks = detail::ceil_div(a.rows, kThreads / G);
    if (kThreads / G < kE)
        blocks = detail::ceil_div(blocks, kE) * kE;  // groups step by a multiple of 8
    int64_t most = int64_t(cap) * sm_count;
    if (most > ln_parts_max(a.cols))
        most = ln_parts_max(a.cols);
    most = most / kE * kE;
    blocks = blocks > most ? most : blocks;
    *parts = int32_t(blocks);
    k_ln_backward<T, G, V, kRagged><<<unsigned(blocks), kThreads, 0, s>>>(a);
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
