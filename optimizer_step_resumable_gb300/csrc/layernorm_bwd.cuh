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
// (A second kernel's many blocks are faster at it than the last block of the
// first: 14.5 against 23.8 us for 8192 x 768 bf16.)  On GB300 65536 x 4096
// bf16 takes 242 us, 6.6 TB/s; 5003 x 1021 float32, whose rows start anywhere,
// 19 us, of which the second kernel and its wait are 5.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "layernorm_dev.cuh"

namespace osr {
namespace {

using namespace ln;

// Blocks an SM keeps resident, and so the registers of a thread: 16 a unit
// hold its column sums, 8 its weights.  Four units want 200 and more: at 128,
// with twice the rows on their way, 1024 columns took 84 us instead of 70
// (65536 rows, bf16), 4096 columns 315 instead of 251.
template <int kGroup, int kUnits>
constexpr int kBackwardBlocks = (kUnits == 1   ? 768
                                 : kUnits <= 3 ? 512
                                               : (kGroup > 256 ? kGroup : 256)) /
                                kBlockThreads<kGroup>;

template <typename T, int kGroup, int kUnits>
using BackwardRing =
    Ring<T, kBlockThreads<kGroup>, kUnits * 8 / kE<T>, 2,
         stages_for(2 * kUnits * 8 * int(sizeof(T)) * kBlockThreads<kGroup>,
                    kBackwardBlocks<kGroup, kUnits>, 144 * 1024, 3)>;

// A thread's column sums to their places in a row of cols floats.
template <typename C, int kVecs, int kPairs>
__device__ __forceinline__ void spread(const C& at, const float2 (&sum)[kVecs][kPairs], float edge,
                                       float* row)
{
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
        if (at.has(v)) {
#pragma unroll
            for (int p = 0; p < kPairs; ++p) {
                row[at.column(v) + 2 * p] = sum[v][p].x;
                row[at.column(v) + 2 * p + 1] = sum[v][p].y;
            }
        }
    if (at.has_edge())
        row[at.edge] = edge;
}

// A row is looked at twice in shared memory, for the sums and for dx, rather
// than kept widened in 16 registers more a unit.
template <typename T, int kGroup, int kUnits, Rows kRows>
__global__ void __launch_bounds__(kBlockThreads<kGroup>, (kBackwardBlocks<kGroup, kUnits>))
    k_ln_backward(LnBackward a)
{
    constexpr int kThreads = kBlockThreads<kGroup>;
    constexpr int kGroups = kThreads / kGroup;
    constexpr int kVecs = kUnits * 8 / kE<T>;
    constexpr int kPairs = kP<T>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(16) unsigned char raw[];
    const BackwardRing<T, kGroup, kUnits> ring{reinterpret_cast<uint4*>(raw)};
    constexpr int kStages = BackwardRing<T, kGroup, kUnits>::kDepth;
    __shared__ float slots[2][2][16];
    int turn = 0;
    const int64_t first = int64_t(blockIdx.x) * kGroups;
    const int64_t groups = int64_t(gridDim.x) * kGroups;
    int64_t r = first + threadIdx.x / kGroup;
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + r * a.dy_stride;
    T* dx = static_cast<T*>(a.dx) + r * a.dx_stride;
    const Columns<T, kGroup, kRows> at(a.cols, threadIdx.x % kGroup, x);
    constexpr int kStride = Columns<T, kGroup, kRows>::kStride;
    x += at.start;  // this thread's first vector of row r
    dy += at.start;
    dx += at.start;
    const int edge = at.edge - at.start;
    const bool dy_cut = is_cut<kRows>(dy);
    const int shift = kRows >= kShifted ? head_of(dx) : 0;  // dx's boundaries after x's
    const int64_t x_step = groups * a.x_stride, dy_step = groups * a.dy_stride,
                  dx_step = groups * a.dx_stride;
    struct Scalars {
        float mean, rstd, x, dy;  // of a row; of this thread's edge element
    };
    Scalars next[kStages];  // [i]: of the row i + 1 turns ahead
    auto fetch = [&](int stage, int ahead, Scalars& s) {
        const T* const xr = x + ahead * x_step;
        const T* const gr = dy + ahead * dy_step;
        const int64_t row = r + ahead * groups;
        s = Scalars{0.0f, 0.0f, 0.0f, 0.0f};
        if (row < a.rows) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
                if (at.has(v)) {
                    ring.copy(stage, 0, v, xr + v * kStride);
                    if (dy_cut)
                        ring.copy(stage, 1, v, gr + v * kStride);
                }
            s.mean = a.mean[row];
            s.rstd = a.rstd[row];
            if (at.has_edge()) {
                s.x = detail::load1(xr + edge);
                s.dy = detail::load1(gr + edge);
            }
        }
        commit_copies();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        fetch(i, i, next[i]);

    float2 w[kVecs][kPairs], dw[kVecs][kPairs], db[kVecs][kPairs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        load_weights<T>(a.weight, a.w_f32, at.column(v), at.has(v), 1.0f, w[v]);
        clear(dw[v]);
        clear(db[v]);
    }
    float we = 0.0f, dwe = 0.0f, dbe = 0.0f;
    if (at.has_edge())
        we = weight_at<T>(a.weight, a.w_f32, at.edge, 1.0f);
    const float inv = 1.0f / float(a.cols);
    int stage = 0;
    for (int64_t block_r = first; block_r < a.rows; block_r += groups) {
        const bool live = r < a.rows;
        fetch(stage == 0 ? kStages - 1 : stage - 1, kStages - 1, next[kStages - 1]);
        const Scalars now = next[0];
#pragma unroll
        for (int i = 0; i + 1 < kStages; ++i)
            next[i] = next[i + 1];
        wait_copies<kStages - 1>();
        // one vector of the row, as x - mean and dy; both are 0 outside the
        // row, and so are all products (rstd may be large)
        auto take = [&](int v, float2(&d)[kPairs], float2(&g)[kPairs]) {
            if (live && at.has(v)) {
                ring.read(stage, 0, v, d);
                if (dy_cut)
                    ring.read(stage, 1, v, g);
                else
                    load_vec<kRows>(dy + v * kStride, false, g);
#pragma unroll
                for (int p = 0; p < kPairs; ++p)
                    d[p] = add2(d[p], both(-now.mean));
            } else {
                clear(d);
                clear(g);
            }
        };
        const float de = at.has_edge() ? now.x - now.mean : 0.0f, ge = now.dy * we;
        dwe += now.dy * (de * now.rstd);
        dbe += now.dy;
        float2 s1 = make_float2(ge, 0.0f), s2 = make_float2(ge * (de * now.rstd), 0.0f);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            float2 d[kPairs], g[kPairs];
            take(v, d, g);
#pragma unroll
            for (int p = 0; p < kPairs; ++p) {
                const float2 xh = mul2(d[p], both(now.rstd));
                dw[v][p] = fma2(g[p], xh, dw[v][p]);
                db[v][p] = add2(g[p], db[v][p]);
                const float2 gw = mul2(g[p], w[v][p]);
                s1 = add2(s1, gw);
                s2 = fma2(gw, xh, s2);
            }
        }
        float s[2] = {s1.x + s1.y, s2.x + s2.y};
        group_sum<kGroup>(s, slots, turn);
        // dx = rstd (dy w - m1 - (x - mean) rstd m2)
        const float m1 = s[0] * inv, slope = -now.rstd * (s[1] * inv);
        if (live) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                float2 d[kPairs], g[kPairs];
                take(v, d, g);
#pragma unroll
                for (int p = 0; p < kPairs; ++p)
                    g[p] = mul2(both(now.rstd),
                                fma2(d[p], both(slope), fma2(g[p], w[v][p], both(-m1))));
                if (kRows >= kShifted && shift)
                    *ring.at(stage, 0, v) = narrow_as<T>(g);
                else if (at.has(v))
                    store_vec(dx + v * kStride, narrow_as<T>(g));
            }
            if (at.has_edge())
                store_one(dx + edge, now.rstd * (de * slope + (ge - m1)));
        }
        if constexpr (kRows >= kShifted) {
            group_barrier<kGroup>();
            if (live && shift)
                store_shifted(at, ring, stage, dx, shift);
            group_barrier<kGroup>();  // before the next copies into this stage
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
        r += groups;
        x += x_step;
        dy += dy_step;
        dx += dx_step;
    }
    wait_copies<0>();
    if (!a.sums)
        return;

    float* const mine = a.partials + int64_t(blockIdx.x) * 2 * a.cols;
    if constexpr (kGroups == 1) {
        spread(at, dw, dwe, mine);
        spread(at, db, dbe, mine + a.cols);
    } else {
        // the block's groups join by columns (their heads may differ), in the
        // memory of the ring
        constexpr int kSpan = kGroup * kUnits * 8;
        static_assert(kGroups * kSpan * 4 <= BackwardRing<T, kGroup, kUnits>::kBytes,
                      "the sums fit the ring");
        float* const part = reinterpret_cast<float*>(raw);
        float* const own = part + threadIdx.x / kGroup * kSpan;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            __syncthreads();
            if (pass == 0)
                spread(at, dw, dwe, own);
            else
                spread(at, db, dbe, own);
            __syncthreads();
            for (int c = threadIdx.x; c < a.cols; c += kThreads) {
                float s = 0.0f;
#pragma unroll
                for (int q = 0; q < kGroups; ++q)
                    s += part[q * kSpan + c];
                mine[pass * a.cols + c] = s;
            }
        }
    }
}

// Rows that do not fit a block's registers.  dx: two looks at each row, the
// second from L2.
constexpr int kWideThreads = 512;

template <typename T>
__global__ void __launch_bounds__(kWideThreads) k_ln_backward_wide(LnBackward a)
{
    __shared__ float slots[2][2][16];
    int turn = 0;
    const int cols = a.cols;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* const x = static_cast<const T*>(a.x) + r * a.x_stride;
        const T* const dy = static_cast<const T*>(a.dy) + r * a.dy_stride;
        T* const dx = static_cast<T*>(a.dx) + r * a.dx_stride;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x; c < cols; c += kWideThreads) {
            const float g = detail::load1(dy + c) * weight_at<T>(a.weight, a.w_f32, c, 1.0f);
            s1 += g;
            s2 += g * (detail::load1(x + c) - mean) * rstd;
        }
        float s[2] = {s1, s2};
        group_sum<kWideThreads>(s, slots, turn);
        const float m1 = s[0] / float(cols), m2 = s[1] / float(cols);
        for (int c = threadIdx.x; c < cols; c += kWideThreads) {
            const float g = detail::load1(dy + c) * weight_at<T>(a.weight, a.w_f32, c, 1.0f);
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

template <typename T, int G, int U, Rows kRows>
int launch_one(const LnBackward& a, int sm_count, int32_t* parts, cudaStream_t s)
{
    constexpr int kThreads = kBlockThreads<G>;
    constexpr int kSmem = BackwardRing<T, G, U>::kBytes;
    auto* const kernel = &k_ln_backward<T, G, U, kRows>;
    static const int cap = resident_blocks(kernel, kThreads, kSmem);
    int64_t most = int64_t(cap) * sm_count;
    if (most > ln_parts_max(a.cols))
        most = ln_parts_max(a.cols);
    const int64_t blocks = row_blocks(a.rows, kThreads / G, most);
    *parts = int32_t(blocks);
    kernel<<<unsigned(blocks), kThreads, kSmem, s>>>(a);
    return int(cudaGetLastError());
}

}  // namespace

template <typename T>
int launch_ln_backward_typed(const LnBackward& a, int sm_count, int32_t* parts, cudaStream_t s)
{
    if (a.cols > kLnRegisterCols) {
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
    const bool aligned = a.cols % kE<T> == 0 && rows_aligned(a.x, a.x_stride, sizeof(T)) &&
                         rows_aligned(a.dy, a.dy_stride, sizeof(T)) &&
                         rows_aligned(a.dx, a.dx_stride, sizeof(T));
    return with_layout(a.cols, aligned, [&](auto layout) {
        constexpr int G = decltype(layout)::kGroup, U = decltype(layout)::kUnits;
        constexpr int R = G > 8 ? G : 16;  // lanes for head and tail
        if (!aligned)
            return !rows_alike(a.x, a.x_stride, a.dy, a.dy_stride, sizeof(T))
                       ? launch_one<T, R, U, kMixed>(a, sm_count, parts, s)
                   : rows_alike(a.x, a.x_stride, a.dx, a.dx_stride, sizeof(T))
                       ? launch_one<T, R, U, kRagged>(a, sm_count, parts, s)
                       : launch_one<T, R, U, kShifted>(a, sm_count, parts, s);
        return a.cols == G * U * 8 ? launch_one<T, G, U, kFull>(a, sm_count, parts, s)
                                   : launch_one<T, G, U, kAligned>(a, sm_count, parts, s);
    });
}

}  // namespace osr
