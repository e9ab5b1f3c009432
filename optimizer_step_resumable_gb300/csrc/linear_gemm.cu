// linear_gemm.cu -- how the linear layer's products are divided into tiles, the
// epilogue of products of few rows, and the kernel that joins the sums of a
// divided inner dimension.
#include "linear_gemm.cuh"

namespace osr {
namespace {

using namespace detail;

// The tile's rows are the product's columns: the lanes of a warp have
// neighbouring columns of one row of the product.
struct SwappedEpilogue {
    using Params = StoreParams;
    static constexpr int kUnroll = 1;
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
            with_activation(o.act, [&](auto act) { activate_all<decltype(act)::value>(v); });
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
// from L2.  Their rows are whole vectors; a thread has one, of four splits at
// a time.
constexpr int kJoinThreads = 256;
struct JoinParams {
    LinearOut o;
    const float* partials;
    int64_t rows, columns;
    int32_t splits;
};
__global__ void __launch_bounds__(kJoinThreads) k_linear_join(const JoinParams p)
{
    wait_before();
    go_ahead();
    const LinearOut o = with_factor(p.o);
    const int64_t vectors = (p.columns + 7) / 8, all = p.rows * vectors;
    for (int64_t i = int64_t(blockIdx.x) * kJoinThreads + threadIdx.x; i < all;
         i += int64_t(gridDim.x) * kJoinThreads) {
        const int64_t row = i / vectors, column = (i - row * vectors) * 8;
        float v[8] = {};
        for (int32_t s = 0; s < p.splits; s += 4) {
            uint32_t w[4][8] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (s + j < p.splits)
                    load32(p.partials + ((s + j) * all + i) * 8, w[j]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    v[c] += __uint_as_float(w[j][c]);
        }
        with_activation(o.act, [&](auto act) {
            constexpr int kAct = decltype(act)::value;
            if (column + 8 <= p.columns) {
                finish_some<kAct>(o, row, column, v);
            } else {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (column + c < p.columns) {
                        float f[1] = {v[c]};
                        finish_some<kAct>(o, row, column + c, f);
                    }
            }
        });
    }
}

int join(const LinearOut& o, const float* partials, int64_t rows, int64_t columns, int32_t splits,
         int sm_count, cudaStream_t stream)
{
    const int64_t want = (rows * ((columns + 7) / 8) + kJoinThreads - 1) / kJoinThreads;
    const int64_t most = int64_t(sm_count) * 8;
    return launch_early(k_linear_join, dim3(unsigned(want < most ? want : most)), kJoinThreads, 0,
                        stream, JoinParams{o, partials, rows, columns, splits});
}

// Microseconds that a pair of blocks takes for a block of the inner dimension
// of a tile of 256 x bn (8192 x 4096 x 8192: 283, 324 and 414 us in tiles of 256,
// 192 and 128 columns, 64 blocks in 14, 19 and 27 turns; few rows of 76 x 256
// outputs, 16 and 32 blocks: 0.21, 0.19 and 0.14 us in tiles of 128, 64 and 32 columns
// with the weight in L2, 0.37 in all of them with the weight from memory, which no
// constant here stands for), and for the start and the last epilogue of a launch (8192 x
// 768 x 768: 15.8, 12.9 and 14.4 us).
double block_us(int bn)
{
    return bn == 256 ? 0.316 : bn == 192 ? 0.27 : bn == 128 ? 0.24 : bn == 64 ? 0.2 : 0.18;
}
double launch_us(int bn) { return 3.0 + 0.016 * bn; }
int64_t inner_blocks(int64_t inner) { return (inner + kGemmInner - 1) / kGemmInner; }
int64_t tiles_of(int64_t m, int64_t n, int bn)
{
    return ((m + kGemmTileM - 1) / kGemmTileM) * ((n + bn - 1) / bn);
}

// The tensor cores cut each addition, by up to 2^-23 of the sum for each 16
// products of equal signs (1.7 x 2^-24 measured, see linear_chain): 16384 in a row
// lose 1.0e-4 of it, which shows in float32.  Chains of at most 16 blocks, 1024
// products, lose 6.5e-6, and between them the sums are rounded (random values, 8192
// products: 1.0e-6 off in the 2-norm, 4.4e-6 in chains of 4096).  Each
// is added in L2: 8192 x 4096 x 8192 into float32 takes 378 us, 328 in chains of 4096
// and 431 in chains of 1365 that the threads read, add to and write back.
// 16-bit outputs have chains as soon as the cut could pass a quarter of their rounding
// (linear_chain); those add up in float32 in the workspace, and the join rounds them
// (2^20 rows of equal signs into a binary16 dweight: 5.8e-4 off at most, 8.0e-4 in one
// go; 65536 x 2048 x 4096 backward 1204 to 1262 us).
int64_t chains_in(const LinearSize& p, int64_t splits)
{
    const int64_t each = (inner_blocks(p.inner) + splits - 1) / splits;
    return (each + p.chain - 1) / p.chain;
}
// Whether the sums go to L2 and back, for a launch to join.
bool joined(const LinearSize& p, int64_t splits)
{
    return splits > 1 || (!p.f32 && chains_in(p, splits) > 1);
}
double join_us(const LinearSize& p, int64_t splits)
{
    return joined(p, splits) ? 4.0 + double(p.rows * p.columns) * double(splits) * 8.0 / 6e6 : 0.0;
}
void finish_plan(const LinearSize& p, LinearPlan* plan)
{
    plan->chains = int32_t(chains_in(p, plan->splits));
    plan->partials =
        joined(p, plan->splits) ? plan->splits * p.rows * ((p.columns + 7) / 8 * 8) : 0;
}

// Deals `n` long items and `m` short ones out to the pairs; the time until all
// are done.
double deal_out(int64_t n, double long_us, int64_t m, double short_us, int64_t pairs,
                GemmDeal* deal)
{
    const int64_t rounds = n / pairs, ahead = n - rounds * pairs;
    const double low = double(rounds) * long_us, high = low + long_us;
    int64_t after = 0, before = 0;
    double best = ahead ? high : low;
    if (m > 0) {
        // `before` goes up until all short ones are dealt out; a pair that is
        // ahead takes as many as end no later, or, where that is enough, one more
        const double even = (double(n) * long_us + double(m) * short_us) / double(pairs);
        int64_t b = int64_t((even - low) / short_us) - 2;
        best = 0.0;
        for (b = b > 0 ? b : 0;; ++b) {
            const double end = low + double(b) * short_us;
            if (best != 0.0 && best <= end)
                break;
            int64_t a = end > high ? int64_t((end - high) / short_us + 1e-9) : 0;
            const bool enough = a * ahead + b * (pairs - ahead) >= m;
            if (!enough)
                a = a < b ? a + 1 : b;
            if (a * ahead + b * (pairs - ahead) < m)
                continue;
            const double over = ahead ? high + double(a) * short_us : 0.0;
            const double us = over > end ? over : end;
            if (best == 0.0 || us < best) {
                best = us;
                after = a;
                before = b;
            }
            if (enough)
                break;
        }
    }
    if (deal)
        *deal = GemmDeal{int32_t(pairs), int32_t(n), int32_t(ahead), int32_t(m), int32_t(after),
                         int32_t(before)};
    return best;
}
// Of a tile of 256 x 256, with what its start and end hold up, and each chain
// after the first.
double item_us(int64_t blocks, int64_t splits, int64_t chains)
{
    const int64_t each = (blocks + splits - 1) / splits;
    return double(each) * block_us(256) + 0.3 + 1.3 * double(chains - 1);
}

StoreProduct store_product(const LinearProduct& p, const LinearPlan& plan, float* partials,
                           int32_t* gave_up)
{
    StoreProduct s{p.a, p.b, GemmShape{}, StoreParams{p.to, p.a.outer, p.b.outer, 0}, GemmSide{}};
    s.s.splits = plan.splits;
    s.s.chains = plan.chains;
    s.s.gave_up = gave_up;
    if (plan.partials) {
        LinearOut sums{};
        sums.out = partials;
        sums.stride = (p.b.outer + 7) / 8 * 8;
        sums.alpha = 1.0f;
        sums.dtype = sums.residual_dtype = ADAMW_DTYPE_F32;
        sums.vectors = 1;
        s.p.o = sums;
        s.p.split_stride = p.a.outer * sums.stride;
    }
    return s;
}
int join_product(const LinearProduct& p, const LinearPlan& plan, const float* partials,
                 int sm_count, void* stream)
{
    if (!plan.partials)
        return cudaSuccess;
    return join(p.to, partials, p.a.outer, p.b.outer, plan.splits, sm_count,
                static_cast<cudaStream_t>(stream));
}

// Gives the sums to the product's launch, unless its few blocks would be long at
// them.
int take_side(const GemmSide* side, int64_t items, int sm_count, StoreProduct* s, void* stream)
{
    if (!side)
        return cudaSuccess;
    const int64_t blocks = 2 * (items < sm_count / 2 ? items : sm_count / 2);
    if (side->columns > 32 * 4 * blocks)
        return launch_linear_bias_grad(*side, stream);
    s->side = *side;
    return cudaSuccess;
}

}  // namespace

LinearPlan linear_plan(const LinearSize& p, int sm_count)
{
    LinearPlan best{};
    if (linear_few_pays(p)) {
        best.few = true;
        best.splits = best.chains = 1;
        return best;
    }
    const bool swapped = p.rows <= 128 && p.rows < p.columns;
    const int64_t m = swapped ? p.columns : p.rows, n = swapped ? p.rows : p.columns;
    const int64_t blocks = inner_blocks(p.inner), pairs = sm_count / 2;
    // rows of fewer than 64 outer elements cannot be copied across
    const int least = swapped && !(p.a_across || n > 64) ? (n > 32 ? 64 : 32) : 128;
    const int widths[] = {least, 192, 256};
    // Time goes by the turns that the busiest pair takes; cutting the inner
    // dimension fills the GPU better.
    double least_us = 0.0;
    for (const int bn : widths) {
        if (bn > least && (swapped || n <= bn - 64))
            continue;
        const int64_t tiles = tiles_of(m, n, bn);
        for (int64_t s = 1; s <= 32 && s <= (blocks + 3) / 4; ++s) {
            const double turns = double((tiles * s + pairs - 1) / pairs);
            const int64_t each = (blocks + s - 1) / s;
            const double us = turns * (double(each) * block_us(bn) +
                                       1.3 * double(chains_in(p, s) - 1)) +
                              launch_us(bn) + join_us(p, s);
            if (best.bn == 0 || us < least_us) {
                least_us = us;
                best.bn = bn;
                best.splits = int32_t(s);
            }
            if (tiles >= 4 * pairs)
                break;  // enough turns
        }
    }
    best.swapped = swapped;
    finish_plan(p, &best);
    return best;
}

double linear_us(const LinearSize& p, const LinearSize* q, int sm_count)
{
    const int64_t pairs = sm_count / 2, n = tiles_of(p.rows, p.columns, 256);
    const double a = item_us(inner_blocks(p.inner), 1, chains_in(p, 1));
    if (!q)
        return launch_us(256) + deal_out(n, a, 0, a, pairs, nullptr);
    const int64_t m = tiles_of(q->rows, q->columns, 256);
    const double b = item_us(inner_blocks(q->inner), 1, chains_in(*q, 1));
    return launch_us(256) + (a >= b ? deal_out(n, a, m, b, pairs, nullptr)
                                    : deal_out(m, b, n, a, pairs, nullptr));
}

bool linear_plan_two(const LinearSize& p, const LinearSize& q, int sm_count, LinearPlan* p_plan,
                     LinearPlan* q_plan)
{
    *p_plan = linear_plan(p, sm_count);
    *q_plan = linear_plan(q, sm_count);
    // tiles of 256 x 256 have to fit both
    if (p_plan->few || p_plan->swapped || p.rows <= 128 || p.columns <= 128 || q.rows <= 128 ||
        q.columns <= 128)
        return false;
    const int64_t pairs = sm_count / 2, blocks[] = {inner_blocks(p.inner), inner_blocks(q.inner)};
    const int64_t tiles[] = {tiles_of(p.rows, p.columns, 256), tiles_of(q.rows, q.columns, 256)};
    static const int kSplits[] = {1, 2, 3, 4, 5, 6, 8, 12, 16, 24};
    int best[2] = {1, 1};
    double least_us = 0.0;
    for (const int s : kSplits) {
        if (s > 1 && (s > (blocks[0] + 3) / 4 || tiles[0] * (s - 1) >= 4 * pairs))
            break;
        for (const int t : kSplits) {
            if (t > 1 && (t > (blocks[1] + 3) / 4 || tiles[1] * (t - 1) >= 4 * pairs))
                break;
            const double a = item_us(blocks[0], s, chains_in(p, s));
            const double b = item_us(blocks[1], t, chains_in(q, t));
            const int64_t n = tiles[0] * s, m = tiles[1] * t;
            const double us = (a >= b ? deal_out(n, a, m, b, pairs, nullptr)
                                      : deal_out(m, b, n, a, pairs, nullptr)) +
                              join_us(p, s) + join_us(q, t);
            if (least_us == 0.0 || us < least_us) {
                least_us = us;
                best[0] = s;
                best[1] = t;
            }
        }
    }
    *p_plan = LinearPlan{false, false, 256, best[0], 1, 0};
    *q_plan = LinearPlan{false, false, 256, best[1], 1, 0};
    finish_plan(p, p_plan);
    finish_plan(q, q_plan);
    return true;
}

int linear_product(const LinearProduct& p, const LinearPlan& plan, float* partials,
                   const GemmSide* side, int sm_count, int32_t* gave_up, void* stream)
{
    if (plan.few) {
        const int e = side ? launch_linear_bias_grad(*side, stream) : int(cudaSuccess);
        return e == cudaSuccess ? linear_few(p, sm_count, stream) : e;
    }
    StoreProduct s = store_product(p, plan, partials, gave_up);
    const int64_t tiles = plan.swapped ? tiles_of(p.b.outer, p.a.outer, plan.bn)
                                       : tiles_of(p.a.outer, p.b.outer, plan.bn);
    int e = take_side(side, tiles * plan.splits, sm_count, &s, stream);
    if (e != cudaSuccess)
        return e;
    if (plan.swapped) {
        const auto run = plan.bn == 32   ? gemm_run<32, SwappedEpilogue>
                         : plan.bn == 64 ? gemm_run<64, SwappedEpilogue>
                                         : gemm_run<128, SwappedEpilogue>;
        e = run(s.b, s.a, s.s, p.bf16, s.p, s.side, sm_count, static_cast<cudaStream_t>(stream));
    } else if (s.p.o.dtype == ADAMW_DTYPE_F32) {
        e = linear_store_f32(plan.bn, s, p.bf16, sm_count, stream);
    } else {
        const bool plain = !s.p.o.bias && !s.p.o.z && s.p.o.act == LINEAR_NONE;
        const auto store =
            s.p.o.dtype == ADAMW_DTYPE_BF16 ? linear_store_bf16 : linear_store_f16;
        e = store(plan.bn, s, plain, p.bf16, sm_count, stream);
    }
    return e == cudaSuccess ? join_product(p, plan, partials, sm_count, stream) : e;
}

int linear_product_two(const LinearProduct& p, const LinearPlan& p_plan, float* p_partials,
                       const LinearProduct& q, const LinearPlan& q_plan, float* q_partials,
                       const GemmSide* side, int sm_count, int32_t* gave_up, void* stream)
{
    StoreProduct a = store_product(p, p_plan, p_partials, gave_up);
    StoreProduct b = store_product(q, q_plan, q_partials, gave_up);
    // the longer items first; an item has the chains of its plan, whatever the type
    // that its sums leave in (by the type, a piece's dx in float32 counted chains that
    // it does not have: 8192 x 768 and 32000 words into a float32 dweight ended at 281
    // us of the model's, where its plan ends at 262)
    const double a_us = item_us(inner_blocks(p.a.inner), p_plan.splits, p_plan.chains);
    const double b_us = item_us(inner_blocks(q.a.inner), q_plan.splits, q_plan.chains);
    const int64_t a_items = tiles_of(p.a.outer, p.b.outer, 256) * p_plan.splits;
    const int64_t b_items = tiles_of(q.a.outer, q.b.outer, 256) * q_plan.splits;
    const int64_t items = a_items + b_items, most = sm_count / 2;
    if (items >= int64_t(1) << 30)
        return int(cudaErrorInvalidValue);
    const int64_t pairs = items < most ? items : most;
    const bool turned = b_us > a_us;
    StoreProduct &first = turned ? b : a, &second = turned ? a : b;
    int e = take_side(side, items, sm_count, &first, stream);
    if (e != cudaSuccess)
        return e;
    GemmDeal deal;
    if (turned)
        deal_out(b_items, b_us, a_items, a_us, pairs, &deal);
    else
        deal_out(a_items, a_us, b_items, b_us, pairs, &deal);
    switch (first.p.o.dtype) {
    case ADAMW_DTYPE_F32: e = linear_store_two_f32(first, second, p.bf16, deal, stream); break;
    case ADAMW_DTYPE_BF16: e = linear_store_two_bf16(first, second, deal, stream); break;
    default: e = linear_store_two_f16(first, second, deal, stream);
    }
    if (e == cudaSuccess)
        e = join_product(p, p_plan, p_partials, sm_count, stream);
    return e == cudaSuccess ? join_product(q, q_plan, q_partials, sm_count, stream) : e;
}

int launch_linear_zero(const LinearOut& to, int64_t rows, int64_t columns, int sm_count,
                       void* stream)
{
    return join(to, nullptr, rows, columns, 0, sm_count, static_cast<cudaStream_t>(stream));
}

}  // namespace osr
