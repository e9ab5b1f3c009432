// cross_entropy_api.cu -- the C ABI entry points of the cross entropy over a
// vocabulary (linear_cross_entropy_* of include/adamw_ckpt.h).
#include <cmath>
#include <cstdint>
#include <new>

#include <cuda_runtime.h>

#include "api_util.h"
#include "arrays.h"
#include "cross_entropy.h"
#include "linear.h"
#include "product_ctx.h"

namespace {

using osr::check_apart;
using osr::check_array;
using osr::check_rows;
using osr::copy_of;
using osr::copy_readable;
using osr::cuda_fail;
using osr::DeviceScope;
using osr::fail;
using osr::gemm_readable;
using osr::GemmOperand;
using osr::kCeColumns;
using osr::kCeParts;
using osr::known_dtype;
using osr::LinearPlan;
using osr::LinearProduct;
using osr::LinearSize;
using osr::on_vectors;
using osr::Pieces;
using osr::rows_of;
using osr::size_of;
using osr::vector_of;
using osr::whole;
using osr::Workspace;

struct Needs {  // without gaps: compared byte by byte
    bool f16, backward, copy_x, copy_weight, in_out, dx, dweight, grad_in_out;
    bool grad_f32, grad_mixed;  // neither float32 nor the other matrices' type
};
int64_t chain_of(bool f16)
{
    return osr::linear_chain(f16 ? ADAMW_DTYPE_F16 : ADAMW_DTYPE_BF16);
}
// How the products of a piece of `columns` are computed.
struct Plans {
    LinearPlan dx{}, dweight{};
    bool together = false;  // in one launch
};
// The pieces that the vocabulary is divided into for the backward pass.
struct Pieced {
    int64_t columns = 0;
    Plans plans, last;  // of the pieces, and of the last, which may be shorter
};

}  // namespace

struct linear_ce_ctx {
    osr::ProductContext base;
    int32_t dim = 0, vocab = 0;
    // the last piece found, which takes as long as some launches
    int64_t piece_rows = -1, piece = 0;
    osr::RecentPlans<Needs, Pieced> pieced;
};

namespace {


constexpr int32_t kMaxDim = 1 << 20, kMaxVocab = 1 << 24;
constexpr int64_t kMaxRows = int64_t(1) << 30;
// The gradient of a piece's logits takes this many bytes at most (or 256
// columns).
constexpr int64_t kPieceBytes = int64_t(256) << 20;

int64_t tiles(int64_t vocab) { return (vocab + kCeColumns - 1) / kCeColumns; }

// last: dx leaves in its own type; before, the sum so far stays in float32.
Plans make_plans(const linear_ce_ctx* c, int64_t rows, int64_t columns, bool last, const Needs& n)
{
    Plans p;
    const int sms = c->base.sm_count;
    const LinearSize dx{rows, c->dim, columns, false, !n.in_out, !last, chain_of(n.f16)};
    const LinearSize dw{n.grad_in_out ? c->dim : columns, n.grad_in_out ? columns : c->dim, rows,
                        true, true, n.grad_f32,
                        n.grad_f32 ? osr::linear_chain(ADAMW_DTYPE_F32)
                                   : chain_of(n.f16 != n.grad_mixed)};
    if (n.dx && n.dweight && !n.grad_mixed) {
        p.together = osr::linear_plan_two(dx, dw, sms, &p.dx, &p.dweight);
    } else {
        if (n.dx)
            p.dx = osr::linear_plan(dx, sms);
        if (n.dweight)
            p.dweight = osr::linear_plan(dw, sms);
    }
    return p;
}

// The time of a piece, as far as it depends on the division, the same for all types.
double piece_us(const linear_ce_ctx* c, int64_t rows, int64_t columns)
{
    const int64_t chain = osr::linear_chain(ADAMW_DTYPE_BF16);
    const LinearSize logits{rows, columns, c->dim, false, false, false, chain};
    const LinearSize dx{rows, c->dim, columns, false, true, false, chain};
    const LinearSize dw{columns, c->dim, rows, true, true, false, chain};
    return osr::linear_us(logits, nullptr, c->base.sm_count) +
           osr::linear_us(dx, &dw, c->base.sm_count);
}

// Columns of a piece, whole tiles.  Tiles of products are as good as they fill
// the pairs of blocks in the end: the number with the least time of all those
// that kPieceBytes allows, down to half of them and not more than 64 tiles fewer
// (8192 x 768 x 32000 backward: 797 us in two equal pieces, 773 so).
int64_t find_piece(const linear_ce_ctx* c, int64_t rows)
{
    const int64_t all = tiles(c->vocab);
    int64_t most = kPieceBytes / (2 * rows) / kCeColumns, best = 0;
    most = most < 1 ? 1 : most > all ? all : most;
    double least_us = 0.0;
    for (int64_t t = most; t >= (most + 1) / 2 && t >= most - 64; --t) {
        const int64_t columns = t * kCeColumns, others = (all - 1) / t;
        const double us = double(others) * piece_us(c, rows, columns) +
                          piece_us(c, rows, c->vocab - others * columns);
        if (best == 0 || us < least_us) {
            least_us = us;
            best = columns;
        }
    }
    return best;
}
int64_t piece_of(linear_ce_ctx* c, int64_t rows)
{
    if (rows != c->piece_rows) {
        c->piece = find_piece(c, rows);
        c->piece_rows = rows;
    }
    return c->piece;
}
Pieced make_pieces(linear_ce_ctx* c, int64_t rows, const Needs& n)
{
    Pieced p;
    p.columns = piece_of(c, rows);
    const int64_t end = c->vocab - (c->vocab - 1) / p.columns * p.columns;
    p.last = make_plans(c, rows, end, true, n);
    p.plans = c->vocab > p.columns ? make_plans(c, rows, p.columns, false, n) : p.last;
    return p;
}
const Pieced& pieces_of(linear_ce_ctx* c, int64_t rows, const Needs& n)
{
    return c->pieced.of(rows, n, [&] { return make_pieces(c, rows, n); });
}

struct Parts {
    void* x = nullptr;
    void* weight = nullptr;
    float2* parts = nullptr;  // forward
    float* at = nullptr;
    float* norms = nullptr;  // backward, binary16
    void* gradient = nullptr;
    float* dx = nullptr;  // the sum over the pieces so far
    float* dx_partials = nullptr;
    float* dweight_partials = nullptr;
};

int64_t larger(int64_t a, int64_t b) { return a > b ? a : b; }

int64_t lay_out(const linear_ce_ctx* c, int64_t rows, const Needs& n, const Pieced& pieced,
                void* memory, Parts* p)
{
    Workspace w(memory);
    if (n.copy_x)
        p->x = w.take(2 * rows * whole(c->dim));
    if (n.copy_weight)
        p->weight = w.take(2 * (n.in_out ? c->dim * whole(c->vocab) : c->vocab * whole(c->dim)));
    if (!n.backward) {
        p->parts = static_cast<float2*>(w.take(8 * rows * kCeParts * tiles(c->vocab)));
        p->at = static_cast<float*>(w.take(4 * rows));
        return w.bytes();
    }
    p->norms = static_cast<float*>(w.take(8));
    p->gradient = w.take(2 * rows * pieced.columns);
    if (n.dx && pieced.columns < c->vocab)
        p->dx = static_cast<float*>(w.take(4 * rows * whole(c->dim)));
    if (const int64_t sums = larger(pieced.plans.dx.partials, pieced.last.dx.partials))
        p->dx_partials = static_cast<float*>(w.take(4 * sums));
    if (const int64_t sums = larger(pieced.plans.dweight.partials, pieced.last.dweight.partials))
        p->dweight_partials = static_cast<float*>(w.take(4 * sums));
    return w.bytes();
}

int check_common(linear_ce_ctx* ctx, int32_t dtype, int64_t rows, int32_t flags, int32_t known)
{
    if (!ctx)
        return fail(ADAMW_EINVAL, "ctx is NULL");
    if (dtype != ADAMW_DTYPE_BF16 && dtype != ADAMW_DTYPE_F16)
        return fail(ADAMW_EINVAL, "dtype=%d is not BF16 or F16", dtype);
    if (rows < 0 || rows > kMaxRows)
        return fail(ADAMW_EINVAL, "rows=%lld outside [0, 2^30]", (long long)rows);
    if (flags & ~known)
        return fail(ADAMW_EINVAL, "unknown flags 0x%x", flags);
    return ADAMW_OK;
}

int64_t high(const linear_ce_ctx* c, bool in_out) { return in_out ? c->dim : c->vocab; }
int32_t wide(const linear_ce_ctx* c, bool in_out) { return in_out ? c->vocab : c->dim; }

}  // namespace

extern "C" {

int linear_cross_entropy_create(int32_t dim, int32_t vocab, linear_ce_ctx** out)
{
    osr::clear_error();
    if (!out)
        return fail(ADAMW_EINVAL, "out is NULL");
    *out = nullptr;
    if (dim < 1 || dim > kMaxDim)
        return fail(ADAMW_EINVAL, "dim=%d outside [1, 2^20]", dim);
    if (vocab < 1 || vocab > kMaxVocab)
        return fail(ADAMW_EINVAL, "vocab=%d outside [1, 2^24]", vocab);
    linear_ce_ctx* c = new (std::nothrow) linear_ce_ctx;
    if (!c)
        return fail(ADAMW_EINVAL, "out of host memory");
    c->dim = dim;
    c->vocab = vocab;
    const int rc = osr::product_create(&c->base);
    if (rc != ADAMW_OK) {
        osr::product_free(&c->base);
        delete c;
        return rc;
    }
    *out = c;
    return ADAMW_OK;
}

int linear_cross_entropy_destroy(linear_ce_ctx* ctx)
{
    osr::clear_error();
    if (ctx) {
        osr::product_free(&ctx->base);
        delete ctx;
    }
    return ADAMW_OK;
}

int linear_cross_entropy_workspace(linear_ce_ctx* ctx, int64_t rows, int32_t flags, int64_t* bytes)
{
    osr::clear_error();
    const int rc = check_common(ctx, ADAMW_DTYPE_BF16, rows, flags,
                                LINEAR_FOR_BACKWARD | LINEAR_FOR_ANY_ADDRESS);
    if (rc != ADAMW_OK)
        return rc;
    if (!bytes)
        return fail(ADAMW_EINVAL, "bytes is NULL");
    *bytes = 0;
    if (rows == 0)
        return ADAMW_OK;
    const bool back = flags & LINEAR_FOR_BACKWARD, any = flags & LINEAR_FOR_ANY_ADDRESS;
    // the most that any layout of the weight and its gradient takes
    for (int layout = 0; layout < 4; ++layout) {
        Needs n{false, back, any, any, (layout & 1) != 0, back, back, (layout & 2) != 0};
        // dx and dweight in one launch, or each on its own; dweight in 16 bits or 32;
        // either 16-bit type, where they differ
        const int forms = !back ? 1 : osr::linear_long(rows, ctx->vocab, 0) ? 8 : 4;
        for (int form = 0; form < forms; ++form) {
            n.grad_mixed = (form & 1) != 0;
            n.grad_f32 = (form & 2) != 0;
            n.f16 = (form & 4) != 0;
            Parts p;
            const int64_t b = lay_out(ctx, rows, n, back ? make_pieces(ctx, rows, n) : Pieced{},
                                      nullptr, &p);
            *bytes = *bytes > b ? *bytes : b;
        }
    }
    return ADAMW_OK;
}

int linear_cross_entropy_forward(linear_ce_ctx* ctx, const void* d_x, int64_t x_stride,
                                 const void* d_weight, int64_t weight_stride, int32_t dtype,
                                 const int64_t* d_target, double z_loss, float* d_loss,
                                 float* d_lse, int64_t rows, int32_t flags, void* d_workspace,
                                 int64_t workspace_bytes, void* stream)
{
    osr::clear_error();
    int rc = check_common(ctx, dtype, rows, flags, LINEAR_IN_OUT);
    if (rc != ADAMW_OK)
        return rc;
    const bool in_out = flags & LINEAR_IN_OUT;
    const int64_t w_rows = high(ctx, in_out);
    const int32_t w_cols = wide(ctx, in_out), dim = ctx->dim;
    if ((rc = check_rows(d_x, x_stride, rows, dim, 2, "d_x")) ||
        (rc = check_rows(d_weight, weight_stride, w_rows, w_cols, 2, "d_weight")) ||
        (rc = check_array(d_target, 8, rows == 0, "d_target")) ||
        (rc = check_array(d_loss, 4, rows == 0, "d_loss")) ||
        (rc = check_array(d_lse, 4, true, "d_lse")))
        return rc;
    if (!std::isfinite(float(z_loss)))
        return fail(ADAMW_EINVAL, "z_loss=%g is not finite", z_loss);
    const Pieces outs[] = {vector_of(d_loss, rows, 4, "d_loss"),
                           vector_of(d_lse, rows, 4, "d_lse")};
    const Pieces ins[] = {rows_of(d_x, x_stride, rows, dim, 2, "d_x"),
                          rows_of(d_weight, weight_stride, w_rows, w_cols, 2, "d_weight"),
                          vector_of(d_target, rows, 8, "d_target")};
    if ((rc = check_apart(outs, ins)))
        return rc;
    if ((rc = osr::product_state(&ctx->base)))
        return rc;
    if (rows == 0)
        return ADAMW_OK;
    Needs n{};
    n.copy_x = !gemm_readable(d_x, rows > 1 ? x_stride : 0);
    n.copy_weight = !gemm_readable(d_weight, w_rows > 1 ? weight_stride : 0);
    n.in_out = in_out;
    Parts p;
    if ((rc = osr::check_workspace(d_workspace, workspace_bytes,
                                   lay_out(ctx, rows, n, Pieced{}, d_workspace, &p), outs,
                                   ins)))
        return rc;
    DeviceScope scope(ctx->base.device);
    int e = copy_readable(copy_of(&d_x, &x_stride, rows, dim, p.x),
                          copy_of(&d_weight, &weight_stride, w_rows, w_cols, p.weight), stream);
    if (e == cudaSuccess)
        e = osr::launch_ce_parts(
            osr::CeForward{GemmOperand{d_x, rows, dim, x_stride, false},
                           GemmOperand{d_weight, ctx->vocab, dim, weight_stride, in_out},
                           dtype == ADAMW_DTYPE_BF16, d_target, p.parts, p.at},
            ctx->base.sm_count, ctx->base.gave_up, stream);
    if (e == cudaSuccess)
        e = osr::launch_ce_join(osr::CeJoin{p.parts, int32_t(kCeParts * tiles(ctx->vocab)), p.at,
                                            d_target, rows, ctx->vocab, float(z_loss), d_loss,
                                            d_lse},
                                stream);
    return e == cudaSuccess ? ADAMW_OK : cuda_fail(cudaError_t(e), "cross entropy launch");
}

int linear_cross_entropy_backward(linear_ce_ctx* ctx, const void* d_x, int64_t x_stride,
                                  const void* d_weight, int64_t weight_stride, int32_t dtype,
                                  const int64_t* d_target, const float* d_lse,
                                  const float* d_dloss, double scale, double z_loss, void* d_dx,
                                  int64_t dx_stride, void* d_dweight, int64_t dweight_stride,
                                  int32_t grad_dtype, int64_t rows, int32_t flags,
                                  void* d_workspace, int64_t workspace_bytes, void* stream)
{
    osr::clear_error();
    int rc = check_common(ctx, dtype, rows, flags,
                          LINEAR_IN_OUT | LINEAR_GRAD_IN_OUT | LINEAR_ACCUMULATE);
    if (rc != ADAMW_OK)
        return rc;
    if (!known_dtype(grad_dtype))
        return fail(ADAMW_EINVAL, "grad_dtype=%d is not F32, BF16 or F16", grad_dtype);
    const bool in_out = flags & LINEAR_IN_OUT, grad_in_out = flags & LINEAR_GRAD_IN_OUT;
    const int64_t w_rows = high(ctx, in_out), g_rows = d_dweight ? high(ctx, grad_in_out) : 0;
    const int64_t w_read = rows ? w_rows : 0;
    const int32_t w_cols = wide(ctx, in_out), g_cols = wide(ctx, grad_in_out);
    const int32_t dim = ctx->dim, vocab = ctx->vocab;
    const int64_t dx_rows = d_dx ? rows : 0;
    const size_t gs = size_of(grad_dtype);
    if ((rc = check_rows(d_x, x_stride, rows, dim, 2, "d_x")) ||
        (rc = check_rows(d_weight, weight_stride, w_read, w_cols, 2, "d_weight")) ||
        (rc = check_array(d_target, 8, rows == 0, "d_target")) ||
        (rc = check_array(d_lse, 4, rows == 0, "d_lse")) ||
        (rc = check_array(d_dloss, 4, true, "d_dloss")) ||
        (rc = check_rows(d_dx, dx_stride, dx_rows, dim, 2, "d_dx")) ||
        (rc = check_rows(d_dweight, dweight_stride, g_rows, g_cols, gs, "d_dweight")))
        return rc;
    if (!std::isfinite(float(z_loss)))
        return fail(ADAMW_EINVAL, "z_loss=%g is not finite", z_loss);
    if (!std::isfinite(float(scale)))
        return fail(ADAMW_EINVAL, "scale=%g is not finite", scale);
    const Pieces outs[] = {rows_of(d_dx, dx_stride, dx_rows, dim, 2, "d_dx"),
                           rows_of(d_dweight, dweight_stride, g_rows, g_cols, gs, "d_dweight")};
    const Pieces ins[] = {rows_of(d_x, x_stride, rows, dim, 2, "d_x"),
                          rows_of(d_weight, weight_stride, w_read, w_cols, 2, "d_weight"),
                          vector_of(d_target, rows, 8, "d_target"),
                          vector_of(d_lse, rows, 4, "d_lse"),
                          vector_of(d_dloss, rows, 4, "d_dloss")};
    if ((rc = check_apart(outs, ins)))
        return rc;
    if ((rc = osr::product_state(&ctx->base)))
        return rc;
    DeviceScope scope(ctx->base.device);
    const int sms = ctx->base.sm_count;
    osr::LinearOut whole_dweight{};
    whole_dweight.out = d_dweight;
    whole_dweight.stride = dweight_stride;
    whole_dweight.dtype = grad_dtype;
    whole_dweight.alpha = float(scale);
    whole_dweight.vectors = on_vectors(d_dweight, dweight_stride, g_rows, gs);
    int e = cudaSuccess;
    if (rows == 0) {
        if (flags & LINEAR_ACCUMULATE)
            osr::accumulate_into(whole_dweight);
        if (d_dweight)
            e = osr::launch_linear_zero(whole_dweight, g_rows, g_cols, sms, stream);
        return e == cudaSuccess ? ADAMW_OK : cuda_fail(cudaError_t(e), "cross entropy launch");
    }
    if (!d_dx && !d_dweight)
        return ADAMW_OK;
    Needs n{};
    n.f16 = dtype == ADAMW_DTYPE_F16;
    n.backward = true;
    n.copy_x = !gemm_readable(d_x, rows > 1 ? x_stride : 0);
    n.copy_weight = !gemm_readable(d_weight, w_rows > 1 ? weight_stride : 0);
    n.in_out = in_out;
    n.dx = d_dx;
    n.dweight = d_dweight;
    n.grad_in_out = grad_in_out;
    n.grad_f32 = grad_dtype == ADAMW_DTYPE_F32;
    n.grad_mixed = !n.grad_f32 && grad_dtype != dtype;
    const Pieced& pieced = pieces_of(ctx, rows, n);
    Parts p;
    if ((rc = osr::check_workspace(d_workspace, workspace_bytes,
                                   lay_out(ctx, rows, n, pieced, d_workspace, &p), outs,
                                   ins)))
        return rc;
    const bool bf16 = dtype == ADAMW_DTYPE_BF16;
    e = copy_readable(copy_of(&d_x, &x_stride, rows, dim, p.x),
                      copy_of(&d_weight, &weight_stride, w_rows, w_cols, p.weight), stream);
    osr::CeFactors f{d_target, d_lse, d_dloss, float(2.0 * z_loss), vocab, nullptr};
    if (e == cudaSuccess && !bf16) {
        e = osr::launch_ce_norm(f, rows, p.norms, stream);
        f.norm = p.norms;
    }
    for (int64_t first = 0; first < vocab && e == cudaSuccess; first += pieced.columns) {
        const int64_t columns = vocab - first < pieced.columns ? vocab - first : pieced.columns;
        const uint16_t* const w =
            static_cast<const uint16_t*>(d_weight) + first * (in_out ? 1 : weight_stride);
        e = osr::launch_ce_gradient(
            osr::CeGradient{GemmOperand{d_x, rows, dim, x_stride, false},
                            GemmOperand{w, columns, dim, weight_stride, in_out}, bf16, f,
                            int32_t(first), p.gradient, pieced.columns},
            sms, ctx->base.gave_up, stream);
        const bool last = first + columns == vocab;
        const Plans& plans = last ? pieced.last : pieced.plans;
        LinearProduct x{}, dw{};
        x.bf16 = dw.bf16 = bf16;
        x.a = GemmOperand{p.gradient, rows, columns, pieced.columns, false};
        x.b = GemmOperand{w, dim, columns, weight_stride, !in_out};
        // the pieces' sum in float32; the last one leaves with it
        x.to.out = last ? d_dx : p.dx;
        x.to.stride = last ? dx_stride : whole(dim);
        x.to.dtype = last ? dtype : ADAMW_DTYPE_F32;
        if (first > 0) {
            x.to.residual = p.dx;
            x.to.residual_stride = whole(dim);
            x.to.residual_dtype = ADAMW_DTYPE_F32;
        }
        x.to.alpha = float(scale);
        x.to.alpha_factor = bf16 ? nullptr : p.norms + 1;
        x.to.vectors = last ? on_vectors(d_dx, dx_stride, rows, 2) : 1;
        const GemmOperand by_vocab{p.gradient, columns, rows, pieced.columns, true};
        const GemmOperand by_dim{d_x, dim, rows, x_stride, true};
        dw.a = grad_in_out ? by_dim : by_vocab;
        dw.b = grad_in_out ? by_vocab : by_dim;
        dw.to = whole_dweight;
        dw.to.out = static_cast<char*>(d_dweight) +
                    int64_t(gs) * first * (grad_in_out ? 1 : dweight_stride);
        dw.to.alpha_factor = x.to.alpha_factor;
        if (flags & LINEAR_ACCUMULATE)
            osr::accumulate_into(dw.to);
        int32_t* const gave_up = ctx->base.gave_up;
        if (e == cudaSuccess && plans.together) {
            e = osr::linear_product_two(x, plans.dx, p.dx_partials, dw, plans.dweight,
                                        p.dweight_partials, nullptr, sms, gave_up, stream);
        } else {
            if (e == cudaSuccess && d_dx)
                e = osr::linear_product(x, plans.dx, p.dx_partials, nullptr, sms, gave_up, stream);
            if (e == cudaSuccess && d_dweight)
                e = osr::linear_product(dw, plans.dweight, p.dweight_partials, nullptr, sms,
                                        gave_up, stream);
        }
    }
    return e == cudaSuccess ? ADAMW_OK : cuda_fail(cudaError_t(e), "cross entropy launch");
}

}  // extern "C"
