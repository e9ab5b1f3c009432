// linear_gemm.cu -- the linear layer's products: epilogues of the tiled
// product, and the kernel that joins the sums of a divided inner dimension.
#include <type_traits>

#include "gemm.cuh"
#include "linear_dev.cuh"

namespace osr {
namespace {

using namespace detail;

struct StoreParams {
    LinearOut o;
    float* partials;  // sums of each split, rows x columns; NULL: finished here
    int64_t rows, columns;
};

__device__ __forceinline__ LinearOut with_factor(const LinearOut& o)
{
    LinearOut r = o;
    if (o.alpha_factor)
        r.alpha *= *o.alpha_factor;
    return r;
}

// C consecutive elements of a row on a 32-byte boundary.
template <int C>
__device__ __forceinline__ void add_row(const void* p, int64_t at, int32_t dtype, float (&v)[C])
{
    uint32_t w[8];
    if (dtype == ADAMW_DTYPE_F32) {
#pragma unroll
        for (int i = 0; i < C; i += 8) {
            load32(static_cast<const float*>(p) + at + i, w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i + j] += __uint_as_float(w[j]);
        }
        return;
    }
    const bool bf16 = dtype == ADAMW_DTYPE_BF16;
#pragma unroll
    for (int i = 0; i < C; i += 16) {
        load32(static_cast<const uint16_t*>(p) + at + i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[i + 2 * j] += widen16(w[j] & 0xFFFFu, bf16);
            v[i + 2 * j + 1] += widen16(w[j] >> 16, bf16);
        }
    }
}
template <int C>
__device__ __forceinline__ void store_row(void* p, int64_t at, int32_t dtype, const float (&v)[C])
{
    uint32_t w[8];
    if (dtype == ADAMW_DTYPE_F32) {
#pragma unroll
        for (int i = 0; i < C; i += 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] = __float_as_uint(v[i + j]);
            store32(static_cast<float*>(p) + at + i, w);
        }
        return;
    }
    const bool bf16 = dtype == ADAMW_DTYPE_BF16;
#pragma unroll
    for (int i = 0; i < C; i += 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = narrow32(v[i + 2 * j], v[i + 2 * j + 1], bf16);
        store32(static_cast<uint16_t*>(p) + at + i, w);
    }
}

// The tile's rows are the product's: a thread has a row's neighbouring
// columns.  Rows on 32-byte boundaries go out from each thread, whole sectors
// at a time; others through shared memory, so that a warp's lanes have
// neighbouring columns of one row.
struct StoreEpilogue {
    using Params = StoreParams;
    int32_t row;
    int32_t split;
    __device__ StoreEpilogue(const Params&, const GemmShape&, int32_t r, const GemmItem& it,
                             int32_t)
        : row(r), split(it.split)
    {
    }
    template <int C>
    __device__ __forceinline__ void chunk(const Params& p, const GemmShape&, int32_t column,
                                          float (&v)[C], float* stage)
    {
        const int lane = threadIdx.x % 32;
        LinearOut o = with_factor(p.o);
        bool whole = column + C <= p.columns && o.vectors;
        if (p.partials) {
            o = LinearOut{};
            o.out = p.partials + split * p.rows * p.columns;
            o.stride = p.columns;
            o.alpha = 1.0f;
            whole = column + C <= p.columns && p.columns % 8 == 0;
        }
        if (whole) {
            if (row >= p.rows)
                return;
#pragma unroll
            for (int i = 0; i < C; ++i)
                v[i] *= o.alpha;
            if (o.bias)
#pragma unroll
                for (int i = 0; i < C; ++i)
                    v[i] += load_as(o.bias, column + i, o.bias_dtype);
            if (o.z)
                store_row(o.z, row * o.z_stride + column, o.dtype, v);
            if (o.act != LINEAR_NONE)
                with_activation(o.act, [&](auto act) {
#pragma unroll
                    for (int i = 0; i < C; ++i)
                        v[i] = activated<decltype(act)::value>(v[i]);
                });
            if (o.residual)
                add_row(o.residual, row * o.residual_stride + column, o.residual_dtype, v);
            const int64_t at = row * o.stride + column;
            if (o.accumulate)
                add_row(o.out, at, o.dtype, v);
            store_row(o.out, at, o.dtype, v);
            return;
        }
        if (column >= p.columns)  // the same for the whole warp
            return;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < C; ++i)
            stage[lane * 33 + i] = v[i];
        __syncwarp();
        const int32_t first = row - lane, mine = column + lane;
        if (lane < C && mine < p.columns)
            with_activation(o.act, [&](auto act) {
#pragma unroll 4
                for (int r = 0; r < 32; ++r)
                    if (first + r < p.rows)
                        finish_one<decltype(act)::value>(o, first + r, mine,
                                                         stage[r * 33 + lane]);
            });
        __syncwarp();
    }
    __device__ void end(const Params&, const GemmShape&) {}
};

// The tile's rows are the product's columns: the lanes of a warp have
// neighbouring columns of one row of the product.
struct SwappedEpilogue {
    using Params = StoreParams;
    int32_t column;
    int32_t split;
    __device__ SwappedEpilogue(const Params&, const GemmShape&, int32_t r, const GemmItem& it,
                               int32_t)
        : column(r), split(it.split)
    {
    }
    template <int C>
    __device__ __forceinline__ void chunk(const Params& p, const GemmShape&, int32_t row,
                                          float (&v)[C], float*)
    {
        if (column >= p.columns || row >= p.rows)
            return;
        if (p.partials) {
            float* const out = p.partials + (split * p.rows + row) * p.columns + column;
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (row + i < p.rows)
                    out[i * p.columns] = v[i];
            return;
        }
        const LinearOut o = with_factor(p.o);
        const int32_t count = int32_t(p.rows - row < C ? p.rows - row : C);
        const float bias = o.bias ? load_as(o.bias, column, o.bias_dtype) : 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i)
            v[i] = v[i] * o.alpha + bias;
        if (o.z)
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (i < count)
                    store_as(o.z, (row + i) * o.z_stride + column, o.dtype, v[i]);
        if (o.act != LINEAR_NONE)
            with_activation(o.act, [&](auto act) {
#pragma unroll
                for (int i = 0; i < C; ++i)
                    v[i] = activated<decltype(act)::value>(v[i]);
            });
        if (o.residual)
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (i < count)
                    v[i] += load_as(o.residual, (row + i) * o.residual_stride + column,
                                    o.residual_dtype);
        if (o.accumulate)
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (i < count)
                    v[i] += load_as(o.out, (row + i) * o.stride + column, o.dtype);
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (i < count)
                store_as(o.out, (row + i) * o.stride + column, o.dtype, v[i]);
    }
    __device__ void end(const Params&, const GemmShape&) {}
};

// out = finish(sum over the splits, in order).
constexpr int kJoinThreads = 256;
template <bool kVector>
__global__ void __launch_bounds__(kJoinThreads) k_linear_join(const StoreParams p, int32_t splits)
{
    wait_before();
    go_ahead();
    const LinearOut o = with_factor(p.o);
    const int64_t each = p.rows * p.columns;
    constexpr int kEach = kVector ? 4 : 1;
    with_activation(o.act, [&](auto act) {
        for (int64_t i = (int64_t(blockIdx.x) * kJoinThreads + threadIdx.x) * kEach; i < each;
             i += int64_t(gridDim.x) * kJoinThreads * kEach) {
            float v[kEach] = {};
            for (int32_t s = 0; s < splits; ++s) {
                const float* const from = p.partials + s * each + i;
                if constexpr (kVector) {
                    const float4 f = __ldcg(reinterpret_cast<const float4*>(from));
                    v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
                } else
                    v[0] += __ldcg(from);
            }
            const int64_t row = i / p.columns, column = i - row * p.columns;
#pragma unroll
            for (int j = 0; j < kEach; ++j)
                finish_one<decltype(act)::value>(o, row, column + j, v[j]);
        }
    });
}

int join(const StoreParams& p, int32_t splits, int sm_count, cudaStream_t stream)
{
    const bool vector = p.columns % 4 == 0;
    const int64_t work = p.rows * p.columns / (vector ? 4 : 1);
    const int64_t want = (work + kJoinThreads - 1) / kJoinThreads, most = int64_t(sm_count) * 8;
    return launch_early(vector ? k_linear_join<true> : k_linear_join<false>,
                        dim3(unsigned(want < most ? want : most)), kJoinThreads, 0, stream, p,
                        splits);
}

template <int BN, typename E>
int run(const GemmOperand& a, const GemmOperand& b, GemmShape s, bool bf16, const StoreParams& p,
        int sm_count, cudaStream_t stream)
{
    CUtensorMap ma, mb;
    int e = gemm_map(a, 128, bf16, &ma);
    if (e == cudaSuccess)
        e = gemm_map(b, BN / 2, bf16, &mb);
    if (e != cudaSuccess)
        return e;
    s.tiles_n = (s.n + BN - 1) / BN;
    s.what = mma_what(bf16, a.across, b.across, kGemmTileM, BN);
    return gemm_launch<BN, E>(ma, mb, s, p, sm_count, stream);
}

}  // namespace

LinearPlan linear_plan(int64_t rows, int64_t columns, int64_t inner, bool a_across, int sm_count)
{
    LinearPlan plan{};
    plan.swapped = rows <= 128 && rows < columns;
    const int64_t m = plan.swapped ? columns : rows, n = plan.swapped ? rows : columns;
    if (plan.swapped)
        // rows of fewer than 64 outer elements cannot be copied across
        plan.bn = a_across || n > 64 ? 128 : n > 32 ? 64 : 32;
    else
        plan.bn = n <= 128 ? 128 : 256;
    const int64_t tiles = ((m + kGemmTileM - 1) / kGemmTileM) * ((n + plan.bn - 1) / plan.bn);
    const int64_t blocks = (inner + kGemmInner - 1) / kGemmInner, pairs = sm_count / 2;
    // Cut the inner dimension if that fills the GPU better: time goes by the
    // turns that the busiest pair takes, each as long as its blocks and a
    // few more for its epilogue; joining costs the partial sums' way to L2
    // and back.
    double best = 0.0;
    plan.splits = 1;
    for (int64_t s = 1; s <= 32 && s <= (blocks + 3) / 4; ++s) {
        const double turns = double((tiles * s + pairs - 1) / pairs);
        const double per_block = 0.27 * plan.bn / 256.0 + 0.03;  // microseconds
        double us = turns * (double((blocks + s - 1) / s) * per_block + 1.0) + 1.0;
        if (s > 1)
            us += 3.0 + double(m) * double(n) * double(s) * 8.0 / 6e6;
        if (s == 1 || us < best) {
            best = us;
            plan.splits = int32_t(s);
        }
    }
    plan.partials = plan.splits > 1 ? plan.splits * rows * columns : 0;
    return plan;
}

int linear_product(const LinearProduct& p, const LinearPlan& plan, float* partials, int sm_count,
                   int32_t* gave_up, void* stream)
{
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t rows = p.a.outer, columns = p.b.outer;
    const StoreParams params{p.to, plan.splits > 1 ? partials : nullptr, rows, columns};
    const GemmOperand &a = plan.swapped ? p.b : p.a, &b = plan.swapped ? p.a : p.b;
    GemmShape s{};
    s.m = int32_t(a.outer);
    s.n = int32_t(b.outer);
    s.tiles_m = (s.m + kGemmTileM - 1) / kGemmTileM;
    s.splits = plan.splits;
    s.blocks = int32_t((p.a.inner + kGemmInner - 1) / kGemmInner);
    s.a_across = a.across;
    s.b_across = b.across;
    s.gave_up = gave_up;
    int e;
    if (plan.swapped)
        e = plan.bn == 32   ? run<32, SwappedEpilogue>(a, b, s, p.bf16, params, sm_count, st)
            : plan.bn == 64 ? run<64, SwappedEpilogue>(a, b, s, p.bf16, params, sm_count, st)
                            : run<128, SwappedEpilogue>(a, b, s, p.bf16, params, sm_count, st);
    else
        e = plan.bn == 128 ? run<128, StoreEpilogue>(a, b, s, p.bf16, params, sm_count, st)
                           : run<256, StoreEpilogue>(a, b, s, p.bf16, params, sm_count, st);
    if (e != cudaSuccess || plan.splits == 1)
        return e;
    return join(params, plan.splits, sm_count, st);
}

int launch_linear_zero(const LinearOut& to, int64_t rows, int64_t columns, int sm_count,
                       void* stream)
{
    return join(StoreParams{to, nullptr, rows, columns}, 0, sm_count,
                static_cast<cudaStream_t>(stream));
}

}  // namespace osr
