// layernorm_fwd.cu -- the layer norm's forward pass, for sm_103a.
//
// "Grow a Language Model: Backprop" (unhomeschool.com), section "Every
// forward op gets a backward twin": k_layernorm_fwd keeps each row's mean and
// variance for the backward pass.  HBM-bound: every element is read once and
// written once.  A first mean, then the differences from it and their squares
// are summed from registers; the differences' sum corrects the mean and the
// variance (statistics_of), so a row whose mean is far larger than its spread
// loses nothing (it costs up to 2% in bf16, 4% in float32).  On GB300 65536 x
// 4096 bf16 takes 167 us, 6.4 TB/s; 8192 x 768 6.4 us and one token 2.7.
#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "layernorm_dev.cuh"

namespace osr {
namespace {

using namespace ln;

// Resident blocks the kernel is compiled for: 24 registers a unit hold a
// thread's weights, biases and elements.
template <int kGroup, int kUnits>
constexpr int kForwardBlocks = (kUnits == 1 ? 768 : 512) / kBlockThreads<kGroup>;

template <typename T, int kGroup, int kUnits>
using ForwardRing =
    Ring<T, kBlockThreads<kGroup>, kUnits * 8 / kE<T>, 1,
         stages_for(kUnits * 8 * int(sizeof(T)) * kBlockThreads<kGroup>,
                    kForwardBlocks<kGroup, kUnits>, 64 * 1024, 3)>;

template <typename T, int kGroup, int kUnits, Rows kRows>
__global__ void __launch_bounds__(kBlockThreads<kGroup>, (kForwardBlocks<kGroup, kUnits>))
    k_ln_forward(LnForward a)
{
    constexpr int kThreads = kBlockThreads<kGroup>;
    constexpr int kGroups = kThreads / kGroup;
    constexpr int kVecs = kUnits * 8 / kE<T>;
    detail::wait_before();
    detail::go_ahead();
    extern __shared__ __align__(16) unsigned char raw[];
    const ForwardRing<T, kGroup, kUnits> ring{reinterpret_cast<uint4*>(raw)};
    constexpr int kStages = ForwardRing<T, kGroup, kUnits>::kDepth;
    __shared__ float slots[2][2][16];
    int turn = 0;
    const int64_t first = int64_t(blockIdx.x) * kGroups;
    const int64_t groups = int64_t(gridDim.x) * kGroups;
    int64_t r = first + threadIdx.x / kGroup;
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
    T* y = static_cast<T*>(a.y) + r * a.y_stride;
    const Columns<T, kGroup, kRows> at(a.cols, threadIdx.x % kGroup, x);
    constexpr int kStride = Columns<T, kGroup, kRows>::kStride;
    x += at.start;  // this thread's first vector of row r
    y += at.start;
    const int edge = at.edge - at.start;
    const int shift = kRows == kShifted ? head_of(y) : 0;  // y's boundaries after x's
    const int64_t x_step = groups * a.x_stride, y_step = groups * a.y_stride;
    auto fetch = [&](int stage, int ahead) {
        const T* const row = x + ahead * x_step;
        if (r + ahead * groups < a.rows) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
                if (at.has(v))
                    ring.copy(stage, 0, v, row + v * kStride);
        }
        commit_copies();
    };
    auto edge_of = [&](const T* row, bool live) {
        return live && at.has_edge() ? detail::load1(row + edge) : 0.0f;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        fetch(i, i);
    float next_edge = edge_of(x, r < a.rows);

    float2 w[kVecs][kP<T>], b[kVecs][kP<T>];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        load_weights<T>(a.weight, a.w_f32, at.column(v), at.has(v), 1.0f, w[v]);
        load_weights<T>(a.bias, a.w_f32, at.column(v), at.has(v), 0.0f, b[v]);
    }
    float we = 0.0f, be = 0.0f;
    if (at.has_edge()) {
        we = weight_at<T>(a.weight, a.w_f32, at.edge, 1.0f);
        be = weight_at<T>(a.bias, a.w_f32, at.edge, 0.0f);
    }
    const float inv = 1.0f / float(a.cols);
    int stage = 0;
    // every thread takes part in every sum: the rows past the end are empty
    for (int64_t block_r = first; block_r < a.rows; block_r += groups) {
        const bool live = r < a.rows;
        fetch(stage == 0 ? kStages - 1 : stage - 1, kStages - 1);
        float fe = next_edge;
        wait_copies<kStages - 1>();
        float2 f[kVecs][kP<T>];
        float2 sums = make_float2(fe, 0.0f);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            if (live && at.has(v))
                ring.read(stage, 0, v, f[v]);
            else
                clear(f[v]);
#pragma unroll
            for (int p = 0; p < kP<T>; ++p)
                sums = add2(sums, f[v][p]);
        }
        const int mine = stage;
        stage = stage + 1 == kStages ? 0 : stage + 1;
        float total[1] = {sums.x + sums.y};
        group_sum<kGroup>(total, slots, turn);
        // asked for after this row's was used: the wait for a load is one for
        // all that the same instruction has asked for
        next_edge = edge_of(x + x_step, r + groups < a.rows);
        const float first_mean = total[0] * inv;
        fe = at.has_edge() ? fe - first_mean : 0.0f;
        float2 squares = make_float2(fe * fe, 0.0f);
        sums = make_float2(fe, 0.0f);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
#pragma unroll
            for (int p = 0; p < kP<T>; ++p)
                f[v][p] = add2(f[v][p], both(-first_mean));
            if (!at.has(v))
                clear(f[v]);
#pragma unroll
            for (int p = 0; p < kP<T>; ++p) {
                sums = add2(sums, f[v][p]);
                squares = fma2(f[v][p], f[v][p], squares);
            }
        }
        float both_sums[2] = {sums.x + sums.y, squares.x + squares.y};
        group_sum<kGroup>(both_sums, slots, turn);
        const Statistics st = statistics_of(first_mean, both_sums, inv, a.eps);
        if (live) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                float2 o[kP<T>];
#pragma unroll
                for (int p = 0; p < kP<T>; ++p)
                    o[p] = fma2(fma2(f[v][p], both(st.rstd), both(st.shift)), w[v][p], b[v][p]);
                if (kRows == kShifted && shift)
                    *ring.at(mine, 0, v) = narrow_as<T>(o);
                else if (at.has(v))
                    store_vec(y + v * kStride, narrow_as<T>(o));
            }
            if (at.has_edge())
                store_one(y + edge, (fe * st.rstd + st.shift) * we + be);
            if (at.lane == 0) {
                if (a.mean)
                    a.mean[r] = st.mean;
                if (a.rstd)
                    a.rstd[r] = st.rstd;
            }
        }
        if constexpr (kRows == kShifted) {
            group_barrier<kGroup>();
            if (live && shift)
                store_shifted(at, ring, mine, y, shift);
            group_barrier<kGroup>();  // before the next copies into this stage
        }
        r += groups;
        x += x_step;
        y += y_step;
    }
}

// Rows that do not fit a block's registers: three looks at the row.
template <typename T>
__global__ void __launch_bounds__(kWideThreads, 2) k_ln_forward_wide(LnForward a)
{
    __shared__ float slots[2][2][16];
    int turn = 0;
    const float inv = 1.0f / float(a.cols);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
        const WideColumns<T> at(a.cols, threadIdx.x, x);
        x += at.start;
        T* const y = static_cast<T*>(a.y) + r * a.y_stride + at.start;
        const int edge = at.edge - at.start;
        float fe = at.has_edge() ? detail::load1(x + edge) : 0.0f;
        float2 sums = make_float2(fe, 0.0f);
        each_vector<T, 4>(at, [&](int, const float2(&f)[1][kP<T>]) {
#pragma unroll
            for (int p = 0; p < kP<T>; ++p)
                sums = add2(sums, f[0][p]);
        }, x);
        float total[1] = {sums.x + sums.y};
        group_sum<kWideThreads>(total, slots, turn);
        const float first_mean = total[0] * inv;
        fe = at.has_edge() ? fe - first_mean : 0.0f;
        float2 squares = make_float2(fe * fe, 0.0f);
        sums = make_float2(fe, 0.0f);
        each_vector<T, 4>(at, [&](int, const float2(&f)[1][kP<T>]) {
#pragma unroll
            for (int p = 0; p < kP<T>; ++p) {
                const float2 d = add2(f[0][p], both(-first_mean));
                sums = add2(sums, d);
                squares = fma2(d, d, squares);
            }
        }, x);
        float both_sums[2] = {sums.x + sums.y, squares.x + squares.y};
        group_sum<kWideThreads>(both_sums, slots, turn);
        const Statistics st = statistics_of(first_mean, both_sums, inv, a.eps);
        const bool y_cut = is_cut<kMixed>(y);
        each_vector<T, 2>(at, [&](int v, const float2(&f)[1][kP<T>]) {
            float2 w[kP<T>], b[kP<T>], o[kP<T>];
            load_weights<T>(a.weight, a.w_f32, at.column(v), true, 1.0f, w);
            load_weights<T>(a.bias, a.w_f32, at.column(v), true, 0.0f, b);
#pragma unroll
            for (int p = 0; p < kP<T>; ++p)
                o[p] = fma2(fma2(add2(f[0][p], both(-first_mean)), both(st.rstd), both(st.shift)),
                            w[p], b[p]);
            store_any(y + v * at.kStride, y_cut, narrow_as<T>(o));
        }, x);
        if (at.has_edge())
            store_one(y + edge, (fe * st.rstd + st.shift) *
                                        weight_at<T>(a.weight, a.w_f32, at.edge, 1.0f) +
                                    weight_at<T>(a.bias, a.w_f32, at.edge, 0.0f));
        if (threadIdx.x == 0) {
            if (a.mean)
                a.mean[r] = st.mean;
            if (a.rstd)
                a.rstd[r] = st.rstd;
        }
    }
}

template <typename T, int G, int U, Rows kRows>
int launch_one(const LnForward& a, int sm_count, std::atomic<int>* known, cudaStream_t s)
{
    constexpr int kThreads = kBlockThreads<G>;
    constexpr int kSmem = ForwardRing<T, G, U>::kBytes;
    auto* const kernel = &k_ln_forward<T, G, U, kRows>;
    int per_sm = 0;
    const cudaError_t e = resident_blocks(kernel, kThreads, kSmem, known[kRows], &per_sm);
    if (e != cudaSuccess)
        return int(e);
    const int64_t blocks = row_blocks(a.rows, kThreads / G, int64_t(per_sm) * sm_count);
    return detail::launch_early(kernel, dim3(unsigned(blocks)), kThreads, kSmem, s, a);
}

template <typename T, int G, int U>
int launch_aligned(const LnForward& a, int sm_count, std::atomic<int>* known, cudaStream_t s)
{
    return a.cols == G * U * 8 ? launch_one<T, G, U, kFull>(a, sm_count, known, s)
                               : launch_one<T, G, U, kAligned>(a, sm_count, known, s);
}
template <typename T, int G, int U>
int launch_ragged(const LnForward& a, int sm_count, std::atomic<int>* known, cudaStream_t s)
{
    return rows_alike(a.x, a.x_stride, a.y, a.y_stride, sizeof(T))
               ? launch_one<T, G, U, kRagged>(a, sm_count, known, s)
               : launch_one<T, G, U, kShifted>(a, sm_count, known, s);
}

template <typename T>
int launch_typed(const LnForward& a, int sm_count, std::atomic<int>* known, cudaStream_t s)
{
    if (a.cols > kLnRegisterCols) {
        const int64_t most = int64_t(sm_count) * 4;
        k_ln_forward_wide<T><<<unsigned(a.rows < most ? a.rows : most), kWideThreads, 0, s>>>(a);
        return int(cudaGetLastError());
    }
    const bool aligned = a.cols % kE<T> == 0 && rows_aligned(a.x, a.x_stride, sizeof(T)) &&
                         rows_aligned(a.y, a.y_stride, sizeof(T));
    // Where the backward pass's layouts are not the forward pass's best.  Four
    // vectors of float32 a thread rather than eight pay where they fill most of
    // the block (us for 65.5M elements, four and eight: 2820 columns 98 and 95,
    // 2980 96 and 96, 3040 89 and 93, 4096 82 and 92; 5000 107 and 81, 6148 108
    // and 94, 7420 101 and 92, 7680 90 and 95, 8192 88 and 94).  Ragged rows of
    // 16-bit types in more groups of fewer threads, which hide the first warp's
    // head and tail: 32768 x 2047 53 and 61 us, 65536 x 1100 75 and 103.
    if constexpr (sizeof(T) == 4) {
        if (aligned && a.cols > 3000 && a.cols <= 4096)
            return launch_aligned<T, 256, 2>(a, sm_count, known, s);
        if (aligned && a.cols > 7500 && a.cols <= 8192)
            return launch_aligned<T, 512, 2>(a, sm_count, known, s);
    } else if (!aligned && a.cols > 1024 && a.cols <= 2048) {
        return launch_ragged<T, 64, 4>(a, sm_count, known, s);
    }
    return with_layout(a.cols, aligned, [&](auto layout) {
        constexpr int G = decltype(layout)::kGroup, U = decltype(layout)::kUnits;
        constexpr int R = G > 8 ? G : 16;  // lanes for head and tail
        return aligned ? launch_aligned<T, G, U>(a, sm_count, known, s)
                       : launch_ragged<T, R, U>(a, sm_count, known, s);
    });
}

}  // namespace

int launch_ln_forward(const LnForward& a, int32_t dtype, int sm_count, LnBlocks& known,
                      void* stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == kDtypeBF16)
        return launch_typed<__nv_bfloat16>(a, sm_count, known.per_sm[dtype], s);
    if (dtype == kDtypeF16)
        return launch_typed<__half>(a, sm_count, known.per_sm[dtype], s);
    return launch_typed<float>(a, sm_count, known.per_sm[dtype], s);
}

}  // namespace osr
