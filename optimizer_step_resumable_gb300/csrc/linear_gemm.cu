// linear_gemm.cu -- how the linear layer's products are divided into tiles, the
// epilogue of products of few rows, and the kernel that joins the sums of a
// divided inner dimension.
#include "linear_gemm.cuh"

namespace osr {
namespace {

using namespace detail;

__device__ __forceinline__ LinearOut with_factor(const LinearOut& o)
{
    LinearOut r = o;
    if (o.alpha_factor)
        r.alpha *= *o.alpha_factor;
    return r;
}

// The tile's rows are the product's columns: the lanes of a warp have
// neighbouring columns of one row of the product.
struct SwappedEpilogue {
    using Params = StoreParams;
    int32_t column;
    int32_t split;
    bool again;  // a later chain
    __device__ SwappedEpilogue(const Params&, const GemmShape&, int32_t r, int32_t, int32_t,
                               const GemmItem& it, int32_t, float*)
        : column(r), split(it.split), again(it.chain > 0)
    {
    }
    template <int C>
    __device__ __forceinline__ void chunk(const Params& p, const GemmShape&, int32_t row, int,
                                          float (&v)[C], float*)
    {
        if (column >= p.columns || row >= p.rows)
            return;
        LinearOut o = with_factor(p.o);
        o.out = static_cast<char*>(o.out) +
                split * p.split_stride * (o.dtype == ADAMW_DTYPE_F32 ? 4 : 2);
        if (again) {
            o.residual = o.out;
            o.residual_stride = o.stride;
            o.residual_dtype = o.dtype;
        }
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
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (i < count)
                store_as(o.out, (row + i) * o.stride + column, o.dtype, v[i]);
    }
    __device__ void end(const Params&, const GemmShape&) {}
};

// out = finish(sum over the splits, in order).  What bounds it: the sums' way
// from L2; a thread has eight neighbouring ones (or one, where rows are not
// whole vectors), of four splits at a time.
constexpr int kJoinThreads = 256;
struct JoinParams {
    LinearOut o;
    const float* partials;
    int64_t rows, columns;
    int32_t splits;
};
template <bool kVector>
__global__ void __launch_bounds__(kJoinThreads) k_linear_join(const JoinParams p)
{
    wait_before();
    go_ahead();
    const LinearOut o = with_factor(p.o);
    const int64_t each = p.rows * p.columns;
    constexpr int kEach = kVector ? 8 : 1;
    for (int64_t i = (int64_t(blockIdx.x) * kJoinThreads + threadIdx.x) * kEach; i < each;
         i += int64_t(gridDim.x) * kJoinThreads * kEach) {
        const int64_t row = i / p.columns, column = i - row * p.columns;
        float v[kEach] = {};
        for (int32_t s = 0; s < p.splits; s += 4) {
            uint32_t w[4][kEach] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (s + j < p.splits) {
                    const float* const from = p.partials + (s + j) * each + i;
                    if constexpr (kVector)
                        load32(from, w[j]);
                    else
                        w[j][0] = __float_as_uint(__ldcg(from));
                }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int c = 0; c < kEach; ++c)
                    v[c] += __uint_as_float(w[j][c]);
        }
        with_activation(o.act, [&](auto act) {
            finish_some<decltype(act)::value, kEach>(o, row, column, v);
        });
    }
}

int join(const LinearOut& o, const float* partials, int64_t rows, int64_t columns, int32_t splits,
         int sm_count, cudaStream_t stream)
{
    const bool vector = columns % 8 == 0;
    const int64_t work = rows * columns / (vector ? 8 : 1);
    const int64_t want = (work + kJoinThreads - 1) / kJoinThreads, most = int64_t(sm_count) * 8;
    return launch_early(vector ? k_linear_join<true> : k_linear_join<false>,
                        dim3(unsigned(want < most ? want : most)), kJoinThreads, 0, stream,
                        JoinParams{o, partials, rows, columns, splits});
}

}  // namespace

namespace {

// Microseconds that a pair of blocks takes for a block of the inner dimension
// of a tile, and for a tile besides.
constexpr double block_us(int bn) { return bn == 256 ? 0.30 : bn == 192 ? 0.24 : bn == 128 ? 0.18 : 0.16; }
constexpr double kTileUs = 0.6;

}  // namespace

LinearPlan linear_plan(int64_t rows, int64_t columns, int64_t inner, bool a_across, bool f32,
                       int sm_count)
{
    LinearPlan best{};
    const bool swapped = rows <= 128 && rows < columns;
    const int64_t m = swapped ? columns : rows, n = swapped ? rows : columns;
    const int64_t blocks = (inner + kGemmInner - 1) / kGemmInner, pairs = sm_count / 2;
    // rows of fewer than 64 outer elements cannot be copied across
    const int least = swapped && !(a_across || n > 64) ? (n > 32 ? 64 : 32) : 128;
    const int widths[] = {least, 192, 256};
    // Time goes by the turns that the busiest pair takes; cutting the inner
    // dimension fills the GPU better, and joining the sums costs their way to
    // L2 and back and a launch.
    double least_us = 0.0;
    for (const int bn : widths) {
        if (bn > least && (swapped || n <= bn - 64))
            continue;
        const int64_t tiles = ((m + kGemmTileM - 1) / kGemmTileM) * ((n + bn - 1) / bn);
        for (int64_t s = 1; s <= 32 && s <= (blocks + 3) / 4; ++s) {
            const double turns = double((tiles * s + pairs - 1) / pairs);
            const double tile = double((blocks + s - 1) / s) * block_us(bn);
            // the last tile's epilogue has nothing beside it
            double us = turns * (tile > kTileUs ? tile : kTileUs) + kTileUs * bn / 128.0;
            if (s > 1)
                us += 3.0 + double(m) * double(n) * double(s) * 8.0 / 6e6;
            if (best.bn == 0 || us < least_us) {
                least_us = us;
                best.bn = bn;
                best.splits = int32_t(s);
            }
        }
    }
    best.swapped = swapped;
    best.partials = best.splits > 1 ? best.splits * rows * columns : 0;
    // The tensor cores cut each addition, by up to 2^-24 of the sum: 16384
    // products in a row lose 2e-5 of it, which shows in float32 and not in 16
    // bits.  Chains of at most 64 blocks, 4096 products, lose a quarter.
    const int64_t each = (blocks + best.splits - 1) / best.splits;
    best.chains = f32 ? int32_t((each + 63) / 64) : 1;
    return best;
}

int linear_product(const LinearProduct& p, const LinearPlan& plan, float* partials, int sm_count,
                   int32_t* gave_up, void* stream)
{
    const int64_t rows = p.a.outer, columns = p.b.outer;
    StoreParams params{p.to, rows, columns, 0};
    if (plan.splits > 1) {
        LinearOut sums{};
        sums.out = partials;
        sums.stride = columns;
        sums.alpha = 1.0f;
        sums.dtype = sums.residual_dtype = ADAMW_DTYPE_F32;
        sums.vectors = columns % 8 == 0;
        params.o = sums;
        params.split_stride = rows * columns;
    }
    GemmShape s{};
    s.splits = plan.splits;
    s.chains = plan.chains;
    s.gave_up = gave_up;
    int e;
    if (plan.swapped) {
        e = plan.bn == 32   ? gemm_run<32, SwappedEpilogue>(p.b, p.a, s, p.bf16, params, sm_count,
                                                            stream)
            : plan.bn == 64 ? gemm_run<64, SwappedEpilogue>(p.b, p.a, s, p.bf16, params, sm_count,
                                                            stream)
                            : gemm_run<128, SwappedEpilogue>(p.b, p.a, s, p.bf16, params, sm_count,
                                                             stream);
    } else {
        const auto store = params.o.dtype == ADAMW_DTYPE_F32    ? linear_store_f32
                           : params.o.dtype == ADAMW_DTYPE_BF16 ? linear_store_bf16
                                                                : linear_store_f16;
        e = store(plan.bn, p.a, p.b, s, p.bf16, params, sm_count, stream);
    }
    if (e != cudaSuccess || plan.splits == 1)
        return e;
    return join(p.to, partials, rows, columns, plan.splits, sm_count,
                static_cast<cudaStream_t>(stream));
}

int launch_linear_zero(const LinearOut& to, int64_t rows, int64_t columns, int sm_count,
                       void* stream)
{
    return join(to, nullptr, rows, columns, 0, sm_count, static_cast<cudaStream_t>(stream));
}

}  // namespace osr
