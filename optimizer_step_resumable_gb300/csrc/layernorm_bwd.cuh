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
// bf16 takes 240 us, 6.7 TB/s; 5003 x 1021 float32, whose rows start anywhere,
// 17 us, of which the second kernel and its wait are 5.
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
    detail::wait_before();
    detail::go_ahead();
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

// Rows that do not fit a block's registers.  dx: two looks at each row.
template <typename T>
__global__ void __launch_bounds__(kWideThreads, 2) k_ln_backward_wide(LnBackward a)
{
    __shared__ float slots[2][2][16];
    int turn = 0;
    const float inv = 1.0f / float(a.cols);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
        const WideColumns<T> at(a.cols, threadIdx.x, x);
        x += at.start;
        const T* const dy = static_cast<const T*>(a.dy) + r * a.dy_stride + at.start;
        T* const dx = static_cast<T*>(a.dx) + r * a.dx_stride + at.start;
        const float mean = a.mean[r], rstd = a.rstd[r];
        const int edge = at.edge - at.start;
        float de = 0.0f, ge = 0.0f;
        if (at.has_edge()) {
            de = detail::load1(x + edge) - mean;
            ge = detail::load1(dy + edge) * weight_at<T>(a.weight, a.w_f32, at.edge, 1.0f);
        }
        float2 s1 = make_float2(ge, 0.0f), s2 = make_float2(ge * (de * rstd), 0.0f);
        each_vector<T, 2>(at, [&](int v, const float2(&f)[2][kP<T>]) {
            float2 w[kP<T>];
            load_weights<T>(a.weight, a.w_f32, at.column(v), true, 1.0f, w);
#pragma unroll
            for (int p = 0; p < kP<T>; ++p) {
                const float2 gw = mul2(f[1][p], w[p]);
                s1 = add2(s1, gw);
                s2 = fma2(gw, mul2(add2(f[0][p], both(-mean)), both(rstd)), s2);
            }
        }, x, dy);
        float s[2] = {s1.x + s1.y, s2.x + s2.y};
        group_sum<kWideThreads>(s, slots, turn);
        const float m1 = s[0] * inv, slope = -rstd * (s[1] * inv);
        const bool dx_cut = is_cut<kMixed>(dx);
        each_vector<T, 2>(at, [&](int v, const float2(&f)[2][kP<T>]) {
            float2 w[kP<T>], o[kP<T>];
            load_weights<T>(a.weight, a.w_f32, at.column(v), true, 1.0f, w);
#pragma unroll
            for (int p = 0; p < kP<T>; ++p)
                o[p] = mul2(both(rstd), fma2(add2(f[0][p], both(-mean)), both(slope),
                                             fma2(f[1][p], w[p], both(-m1))));
            store_any(dx + v * at.kStride, dx_cut, narrow_as<T>(o));
        }, x, dy);
        if (at.has_edge())
            store_one(dx + edge, rstd * (de * slope + (ge - m1)));
    }
}

// The column sums of such rows: a vector of columns per thread; strip q of the
// rows (the grid's second dimension) is q, q + 32, ..., whose vectors are the
// same, as 32 is a multiple of kRowStep.
constexpr int kColumnThreads = 128, kAtOnce = 4;  // rows on their way

template <typename T>
__global__ void __launch_bounds__(kColumnThreads) k_ln_columns_wide(LnBackward a)
{
    detail::go_ahead();
    const int vector = blockIdx.x * kColumnThreads + threadIdx.x;
    const int64_t first = blockIdx.y;
    const T* x = static_cast<const T*>(a.x) + first * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + first * a.dy_stride;
    const Columns<T, 1, kMixed> at(a.cols, vector, x);  // vector 0 of lane `vector`
    float* const mine = a.partials + first * 2 * a.cols;
    const int64_t x_step = kLnWideParts * a.x_stride, dy_step = kLnWideParts * a.dy_stride;
    if (at.has(0)) {
        const T* const dy0 = dy + at.start;
        const T* const x0 = x + at.start;
        const bool dy_cut = is_cut<kMixed>(dy0);
        float2 dw[kP<T>], db[kP<T>];
        clear(dw);
        clear(db);
        int64_t i = 0;  // rows done
        for (int64_t r = first; r < a.rows; r += kAtOnce * kLnWideParts, i += kAtOnce) {
            float2 f[kAtOnce][kP<T>], g[kAtOnce][kP<T>];
            float mean[kAtOnce], rstd[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int64_t row = r + u * kLnWideParts;
                if (row < a.rows) {
                    load_vec<kMixed>(x0 + (i + u) * x_step, true, f[u]);
                    load_vec<kMixed>(dy0 + (i + u) * dy_step, dy_cut, g[u]);
                    mean[u] = a.mean[row];
                    rstd[u] = a.rstd[row];
                } else {
                    clear(f[u]);
                    clear(g[u]);
                    mean[u] = rstd[u] = 0.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
                for (int p = 0; p < kP<T>; ++p) {
                    const float2 d = add2(f[u][p], both(-mean[u]));
                    dw[p] = fma2(g[u][p], mul2(d, both(rstd[u])), dw[p]);
                    db[p] = add2(g[u][p], db[p]);
                }
        }
#pragma unroll
        for (int p = 0; p < kP<T>; ++p) {
            mine[at.start + 2 * p] = dw[p].x;
            mine[at.start + 2 * p + 1] = dw[p].y;
            mine[a.cols + at.start + 2 * p] = db[p].x;
            mine[a.cols + at.start + 2 * p + 1] = db[p].y;
        }
    }
    if (at.has_edge()) {
        float dw = 0.0f, db = 0.0f;
        const T* xe = x + at.edge;
        const T* ge = dy + at.edge;
        for (int64_t r = first; r < a.rows; r += kLnWideParts, xe += x_step, ge += dy_step) {
            const float g = detail::load1(ge);
            dw += g * ((detail::load1(xe) - a.mean[r]) * a.rstd[r]);
            db += g;
        }
        mine[at.edge] = dw;
        mine[a.cols + at.edge] = db;
    }
}

template <typename T, int G, int U, Rows kRows>
int launch_one(const LnBackward& a, int sm_count, std::atomic<int>* known, int32_t* parts,
               cudaStream_t s)
{
    constexpr int kThreads = kBlockThreads<G>;
    constexpr int kSmem = BackwardRing<T, G, U>::kBytes;
    auto* const kernel = &k_ln_backward<T, G, U, kRows>;
    int per_sm = 0;
    const cudaError_t e = resident_blocks(kernel, kThreads, kSmem, known[kRows], &per_sm);
    if (e != cudaSuccess)
        return int(e);
    int64_t most = int64_t(per_sm) * sm_count;
    if (most > ln_parts_max(a.cols))
        most = ln_parts_max(a.cols);
    const int64_t blocks = row_blocks(a.rows, kThreads / G, most);
    *parts = int32_t(blocks);
    return detail::launch_early(kernel, dim3(unsigned(blocks)), kThreads, kSmem, s, a);
}

}  // namespace

template <typename T>
int launch_ln_backward_typed(const LnBackward& a, int sm_count, std::atomic<int>* known,
                             int32_t* parts, cudaStream_t s)
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
            <<<dim3(unsigned(detail::ceil_div(a.cols, kColumnThreads * kE<T>)), unsigned(*parts)),
               kColumnThreads, 0, s>>>(a);
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
                       ? launch_one<T, R, U, kMixed>(a, sm_count, known, parts, s)
                   : rows_alike(a.x, a.x_stride, a.dx, a.dx_stride, sizeof(T))
                       ? launch_one<T, R, U, kRagged>(a, sm_count, known, parts, s)
                       : launch_one<T, R, U, kShifted>(a, sm_count, known, parts, s);
        return a.cols == G * U * 8 ? launch_one<T, G, U, kFull>(a, sm_count, known, parts, s)
                                   : launch_one<T, G, U, kAligned>(a, sm_count, known, parts, s);
    });
}

}  // namespace osr
