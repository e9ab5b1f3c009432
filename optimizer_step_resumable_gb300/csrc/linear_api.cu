// linear_api.cu -- the C ABI entry points of the linear layer (linear_* of
// include/adamw_ckpt.h).
#include <cstdint>
#include <new>

#include <cuda_runtime.h>

#include "api_util.h"
#include "arrays.h"
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
using osr::known_dtype;
using osr::linear_chain;
using osr::LinearCopy;
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
    bool f16, backward, copy_x, copy_weight, dz;
    bool in_out;  // the weight, for its copy
    bool dx, dweight, dbias;
    bool grad_in_out, grad_f32, grad_mixed;  // neither float32 nor the other matrices' type
};
// How a call is computed; a function of the sizes and needs.
struct Plans {
    LinearPlan forward{}, dx{}, dweight{};
    bool together = false;  // dx and dweight in one launch
    int32_t strips = 0;
};

}  // namespace

struct linear_ctx {
    osr::ProductContext base;
    int32_t in = 0, out = 0;
    osr::RecentPlans<Needs, Plans> plans;
};

namespace {


constexpr int32_t kMaxFeatures = 1 << 24;
constexpr int64_t kMaxRows = int64_t(1) << 30;

int64_t chain_of(bool f16) { return linear_chain(f16 ? ADAMW_DTYPE_F16 : ADAMW_DTYPE_BF16); }

Plans make_plans(const linear_ctx* c, int64_t rows, const Needs& n)
{
    Plans p;
    const int sms = c->base.sm_count;
    if (!n.backward) {
        p.forward = osr::linear_plan(
            LinearSize{rows, c->out, c->in, false, n.in_out, false, chain_of(n.f16)}, sms);
        return p;
    }
    const LinearSize dx{rows, c->in, c->out, false, !n.in_out, false, chain_of(n.f16)};
    const LinearSize dw{n.grad_in_out ? c->in : c->out, n.grad_in_out ? c->out : c->in, rows, true,
                        true, n.grad_f32,
                        n.grad_f32 ? linear_chain(ADAMW_DTYPE_F32) : chain_of(n.f16 != n.grad_mixed)};
    if (n.dx && n.dweight && !n.grad_mixed) {
        p.together = osr::linear_plan_two(dx, dw, sms, &p.dx, &p.dweight);
    } else {
        if (n.dx)
            p.dx = osr::linear_plan(dx, sms);
        if (n.dweight)
            p.dweight = osr::linear_plan(dw, sms);
    }
    if (n.dbias)
        p.strips = osr::linear_strips(rows, c->out, sms);
    return p;
}

const Plans& plans_of(linear_ctx* c, int64_t rows, const Needs& n)
{
    return c->plans.of(rows, n, [&] { return make_plans(c, rows, n); });
}

// Where the parts of a call's workspace lie; NULL where the call needs none.
struct Parts {
    void* x = nullptr;
    void* weight = nullptr;
    void* dy = nullptr;  // dz, or a copy of dy
    float* partials = nullptr;
    float* dweight_partials = nullptr;
    float* sums = nullptr;
};
int64_t lay_out(const linear_ctx* c, int64_t rows, const Needs& n, const Plans& plans,
                void* memory, Parts* p)
{
    Workspace w(memory);
    if (n.copy_x)
        p->x = w.take(2 * rows * whole(c->in));
    if (n.copy_weight)
        p->weight = w.take(2 * (n.in_out ? c->in * whole(c->out) : c->out * whole(c->in)));
    if (n.dz)
        p->dy = w.take(2 * rows * whole(c->out));
    if (n.dbias)
        p->sums = static_cast<float*>(w.take(4 * int64_t(plans.strips) * c->out));
    const int64_t sums = n.backward ? plans.dx.partials : plans.forward.partials;
    if (sums)
        p->partials = static_cast<float*>(w.take(4 * sums));
    if (plans.dweight.partials)
        p->dweight_partials = static_cast<float*>(w.take(4 * plans.dweight.partials));
    return w.bytes();
}

int check_common(linear_ctx* ctx, int32_t dtype, int32_t activation, int64_t rows, int32_t flags,
                 int32_t known)
{
    if (!ctx)
        return fail(ADAMW_EINVAL, "ctx is NULL");
    if (dtype != ADAMW_DTYPE_BF16 && dtype != ADAMW_DTYPE_F16)
        return fail(ADAMW_EINVAL, "dtype=%d is not BF16 or F16", dtype);
    if (activation < LINEAR_NONE || activation > LINEAR_SILU)
        return fail(ADAMW_EINVAL, "activation=%d is unknown", activation);
    if (rows < 0 || rows > kMaxRows)
        return fail(ADAMW_EINVAL, "rows=%lld outside [0, 2^30]", (long long)rows);
    if (flags & ~known)
        return fail(ADAMW_EINVAL, "unknown flags 0x%x", flags);
    return ADAMW_OK;
}

// Rows of the weight as they lie in memory.
int64_t high(const linear_ctx* c, bool in_out) { return in_out ? c->in : c->out; }
int32_t wide(const linear_ctx* c, bool in_out) { return in_out ? c->out : c->in; }

}  // namespace

extern "C" {

int linear_create(int32_t in_features, int32_t out_features, linear_ctx** out)
{
    osr::clear_error();
    if (!out)
        return fail(ADAMW_EINVAL, "out is NULL");
    *out = nullptr;
    if (in_features < 1 || in_features > kMaxFeatures)
        return fail(ADAMW_EINVAL, "in_features=%d outside [1, 2^24]", in_features);
    if (out_features < 1 || out_features > kMaxFeatures)
        return fail(ADAMW_EINVAL, "out_features=%d outside [1, 2^24]", out_features);
    if (int64_t(in_features) * out_features >= int64_t(1) << 40)
        return fail(ADAMW_EINVAL, "in_features x out_features is 2^40 or more");
    linear_ctx* c = new (std::nothrow) linear_ctx;
    if (!c)
        return fail(ADAMW_EINVAL, "out of host memory");
    c->in = in_features;
    c->out = out_features;
    const int rc = osr::product_create(&c->base);
    if (rc != ADAMW_OK) {
        osr::product_free(&c->base);
        delete c;
        return rc;
    }
    *out = c;
    return ADAMW_OK;
}

int linear_destroy(linear_ctx* ctx)
{
    osr::clear_error();
    if (ctx) {
        osr::product_free(&ctx->base);
        delete ctx;
    }
    return ADAMW_OK;
}

int linear_workspace(linear_ctx* ctx, int64_t rows, int32_t flags, int64_t* bytes)
{
    osr::clear_error();
    const int rc = check_common(ctx, ADAMW_DTYPE_BF16, LINEAR_NONE, rows, flags,
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
        Needs n{false, back, any, any, back, (layout & 1) != 0, back, back, back, (layout & 2) != 0};
        // dx and dweight in one launch, or each on its own; dweight in 16 bits or 32;
        // either 16-bit type, where they differ
        for (int form = 0; form < (osr::linear_long(rows, ctx->in, ctx->out) ? 8 : 4); ++form) {
            n.grad_mixed = (form & 1) != 0;
            n.grad_f32 = (form & 2) != 0;
            n.f16 = (form & 4) != 0;
            if (!back && (n.grad_mixed || n.grad_f32))
                continue;
            Parts p;
            const int64_t b = lay_out(ctx, rows, n, make_plans(ctx, rows, n), nullptr, &p);
            *bytes = *bytes > b ? *bytes : b;
        }
    }
    return ADAMW_OK;
}

int linear_forward(linear_ctx* ctx, const void* d_x, int64_t x_stride, const void* d_weight,
                   int64_t weight_stride, int32_t dtype, const void* d_bias, int32_t bias_dtype,
                   const void* d_residual, int64_t residual_stride, int32_t activation, void* d_y,
                   int64_t y_stride, void* d_z, int64_t z_stride, int64_t rows, int32_t flags,
                   void* d_workspace, int64_t workspace_bytes, void* stream)
{
    osr::clear_error();
    int rc = check_common(ctx, dtype, activation, rows, flags, LINEAR_IN_OUT);
    if (rc != ADAMW_OK)
        return rc;
    if (bias_dtype != ADAMW_DTYPE_F32 && bias_dtype != dtype)
        return fail(ADAMW_EINVAL, "bias_dtype=%d is neither F32 nor dtype=%d", bias_dtype, dtype);
    const bool in_out = flags & LINEAR_IN_OUT;
    const int64_t w_rows = high(ctx, in_out);
    const int32_t w_cols = wide(ctx, in_out), in = ctx->in, out = ctx->out;
    const int64_t z_rows = d_z ? rows : 0, r_rows = d_residual ? rows : 0;
    if ((rc = check_rows(d_x, x_stride, rows, in, 2, "d_x")) ||
        (rc = check_rows(d_weight, weight_stride, w_rows, w_cols, 2, "d_weight")) ||
        (rc = check_array(d_bias, size_of(bias_dtype), true, "d_bias")) ||
        (rc = check_rows(d_residual, residual_stride, r_rows, out, 2, "d_residual")) ||
        (rc = check_rows(d_y, y_stride, rows, out, 2, "d_y")) ||
        (rc = check_rows(d_z, z_stride, z_rows, out, 2, "d_z")))
        return rc;
    const bool in_place = d_residual == d_y && (residual_stride == y_stride || rows <= 1);
    const Pieces outs[] = {rows_of(d_y, y_stride, rows, out, 2, "d_y"),
                           rows_of(d_z, z_stride, z_rows, out, 2, "d_z")};
    const Pieces ins[] = {rows_of(d_x, x_stride, rows, in, 2, "d_x"),
                          rows_of(d_weight, weight_stride, w_rows, w_cols, 2, "d_weight"),
                          vector_of(d_bias, out, size_of(bias_dtype), "d_bias"),
                          rows_of(d_residual, residual_stride, in_place ? 0 : r_rows, out, 2,
                                  "d_residual")};
    if ((rc = check_apart(outs, ins)))
        return rc;
    if ((rc = osr::product_state(&ctx->base)))
        return rc;
    if (rows == 0)
        return ADAMW_OK;
    Needs n{};
    n.f16 = dtype == ADAMW_DTYPE_F16;
    n.copy_x = !gemm_readable(d_x, rows > 1 ? x_stride : 0);
    n.copy_weight = !gemm_readable(d_weight, w_rows > 1 ? weight_stride : 0);
    n.in_out = in_out;
    const Plans& plans = plans_of(ctx, rows, n);
    Parts p;
    if ((rc = osr::check_workspace(d_workspace, workspace_bytes,
                                   lay_out(ctx, rows, n, plans, d_workspace, &p), outs,
                                   ins)))
        return rc;
    DeviceScope scope(ctx->base.device);
    int e = copy_readable(copy_of(&d_x, &x_stride, rows, in, p.x),
                          copy_of(&d_weight, &weight_stride, w_rows, w_cols, p.weight), stream);
    if (e != cudaSuccess)
        return cuda_fail(cudaError_t(e), "linear layer launch");
    LinearProduct m{};
    m.a = GemmOperand{d_x, rows, in, x_stride, false};
    m.b = GemmOperand{d_weight, out, in, weight_stride, in_out};
    m.bf16 = dtype == ADAMW_DTYPE_BF16;
    m.to.out = d_y;
    m.to.stride = y_stride;
    m.to.dtype = dtype;
    m.to.bias = d_bias;
    m.to.bias_dtype = bias_dtype;
    m.to.residual = d_residual;
    m.to.residual_stride = residual_stride;
    m.to.residual_dtype = dtype;
    m.to.z = d_z;
    m.to.z_stride = z_stride;
    m.to.act = activation;
    m.to.alpha = 1.0f;
    m.to.vectors = on_vectors(d_y, y_stride, rows, 2) &&
                   (!d_residual || on_vectors(d_residual, residual_stride, rows, 2)) &&
                   (!d_z || on_vectors(d_z, z_stride, rows, 2));
    e = osr::linear_product(m, plans.forward, p.partials, nullptr, ctx->base.sm_count,
                            ctx->base.gave_up, stream);
    return e == cudaSuccess ? ADAMW_OK : cuda_fail(cudaError_t(e), "linear layer launch");
}

int linear_backward(linear_ctx* ctx, const void* d_dy, int64_t dy_stride, const void* d_x,
                    int64_t x_stride, const void* d_weight, int64_t weight_stride, int32_t dtype,
                    const void* d_z, int64_t z_stride, int32_t activation, void* d_dx,
                    int64_t dx_stride, void* d_dweight, int64_t dweight_stride, void* d_dbias,
                    int32_t grad_dtype, int64_t rows, int32_t flags, void* d_workspace,
                    int64_t workspace_bytes, void* stream)
{
    osr::clear_error();
    int rc = check_common(ctx, dtype, activation, rows, flags,
                          LINEAR_IN_OUT | LINEAR_GRAD_IN_OUT | LINEAR_ACCUMULATE);
    if (rc != ADAMW_OK)
        return rc;
    if (!known_dtype(grad_dtype))
        return fail(ADAMW_EINVAL, "grad_dtype=%d is not F32, BF16 or F16", grad_dtype);
    const bool in_out = flags & LINEAR_IN_OUT, grad_in_out = flags & LINEAR_GRAD_IN_OUT;
    const bool accumulate = flags & LINEAR_ACCUMULATE, act = activation != LINEAR_NONE;
    const int64_t w_rows = high(ctx, in_out), g_rows = d_dweight ? high(ctx, grad_in_out) : 0;
    const int32_t w_cols = wide(ctx, in_out), g_cols = wide(ctx, grad_in_out);
    const int32_t in = ctx->in, out = ctx->out;
    const int64_t z_rows = act ? rows : 0, dx_rows = d_dx ? rows : 0;
    // the weight is read for dx, x for dweight
    const int64_t w_read = d_dx && rows ? w_rows : 0, x_read = d_dweight ? rows : 0;
    const size_t gs = size_of(grad_dtype);
    if ((rc = check_rows(d_dy, dy_stride, rows, out, 2, "d_dy")) ||
        (rc = check_rows(d_x, x_stride, x_read, in, 2, "d_x")) ||
        (rc = check_rows(d_weight, weight_stride, w_read, w_cols, 2, "d_weight")) ||
        (rc = check_rows(d_z, z_stride, z_rows, out, 2, "d_z")) ||
        (rc = check_rows(d_dx, dx_stride, dx_rows, in, 2, "d_dx")) ||
        (rc = check_rows(d_dweight, dweight_stride, g_rows, g_cols, gs, "d_dweight")) ||
        (rc = check_array(d_dbias, gs, true, "d_dbias")))
        return rc;
    const Pieces outs[] = {rows_of(d_dx, dx_stride, dx_rows, in, 2, "d_dx"),
                           rows_of(d_dweight, dweight_stride, g_rows, g_cols, gs, "d_dweight"),
                           vector_of(d_dbias, out, gs, "d_dbias")};
    const Pieces ins[] = {rows_of(d_dy, dy_stride, rows, out, 2, "d_dy"),
                          rows_of(d_x, x_stride, x_read, in, 2, "d_x"),
                          rows_of(d_weight, weight_stride, w_read, w_cols, 2, "d_weight"),
                          rows_of(d_z, z_stride, z_rows, out, 2, "d_z")};
    if ((rc = check_apart(outs, ins)))
        return rc;
    if ((rc = osr::product_state(&ctx->base)))
        return rc;
    DeviceScope scope(ctx->base.device);
    const int sms = ctx->base.sm_count;
    Needs n{};
    n.f16 = dtype == ADAMW_DTYPE_F16;
    n.backward = true;
    n.copy_x = x_read && !gemm_readable(d_x, rows > 1 ? x_stride : 0);
    n.copy_weight = w_read && !gemm_readable(d_weight, w_rows > 1 ? weight_stride : 0);
    n.in_out = in_out;
    n.grad_in_out = grad_in_out;
    n.grad_f32 = grad_dtype == ADAMW_DTYPE_F32;
    n.grad_mixed = !n.grad_f32 && grad_dtype != dtype;
    n.dx = dx_rows;
    n.dweight = d_dweight && rows;
    n.dbias = d_dbias && rows;
    n.dz = rows && (d_dx || d_dweight) && (act || !gemm_readable(d_dy, rows > 1 ? dy_stride : 0));
    const Plans none, &plans = rows ? plans_of(ctx, rows, n) : none;
    Parts p;
    if ((rc = osr::check_workspace(d_workspace, workspace_bytes,
                                   lay_out(ctx, rows, n, plans, d_workspace, &p), outs,
                                   ins)))
        return rc;
    const LinearCopy weight_copy = copy_of(&d_weight, &weight_stride, w_rows, w_cols, p.weight);
    const LinearCopy x_copy = copy_of(&d_x, &x_stride, rows, in, p.x);
    int e = cudaSuccess;
    if (n.dz || n.dbias) {
        osr::LinearSlope s{};
        s.dy = d_dy;
        s.dy_stride = dy_stride;
        s.z = d_z;
        s.z_stride = z_stride;
        s.act = activation;
        s.bf16 = dtype == ADAMW_DTYPE_BF16;
        s.dz = p.dy;
        s.stride = whole(out);
        s.rows = rows;
        s.columns = out;
        s.partials = p.sums;
        s.strips = n.dbias ? plans.strips : osr::linear_strips(rows, out, sms);
        s.copies[0] = weight_copy;
        s.copies[1] = x_copy;
        e = osr::launch_linear_slope(s, stream);
    } else {
        e = copy_readable(weight_copy, x_copy, stream);
    }
    const osr::GemmSide bias{p.sums,  n.dbias ? plans.strips : 0, out, d_dbias, grad_dtype,
                             accumulate};
    const osr::GemmSide* side = n.dbias ? &bias : nullptr;
    if (e == cudaSuccess && d_dbias && (rows == 0 || (!n.dx && !n.dweight)))
        e = osr::launch_linear_bias_grad(bias, stream);
    if (e != cudaSuccess)
        return cuda_fail(cudaError_t(e), "linear layer launch");
    const void* dz = n.dz ? p.dy : d_dy;
    const int64_t dz_stride = n.dz ? whole(out) : dy_stride;
    LinearProduct x{}, w{};  // of dx and dweight
    x.bf16 = w.bf16 = dtype == ADAMW_DTYPE_BF16;
    x.a = GemmOperand{dz, rows, out, dz_stride, false};
    x.b = GemmOperand{d_weight, in, out, weight_stride, !in_out};
    x.to.out = d_dx;
    x.to.stride = dx_stride;
    x.to.dtype = dtype;
    x.to.alpha = 1.0f;
    x.to.vectors = on_vectors(d_dx, dx_stride, rows, 2);
    const GemmOperand by_out{dz, out, rows, dz_stride, true}, by_in{d_x, in, rows, x_stride, true};
    w.a = grad_in_out ? by_in : by_out;
    w.b = grad_in_out ? by_out : by_in;
    w.to.out = d_dweight;
    w.to.stride = dweight_stride;
    w.to.dtype = grad_dtype;
    w.to.alpha = 1.0f;
    w.to.vectors = on_vectors(d_dweight, dweight_stride, g_rows, gs);
    if (accumulate)
        osr::accumulate_into(w.to);
    int32_t* const gave_up = ctx->base.gave_up;
    if (plans.together) {
        e = osr::linear_product_two(x, plans.dx, p.partials, w, plans.dweight, p.dweight_partials,
                                    side, sms, gave_up, stream);
    } else {
        if (n.dx)
            e = osr::linear_product(x, plans.dx, p.partials, side, sms, gave_up, stream);
        if (e == cudaSuccess && n.dweight)
            e = osr::linear_product(w, plans.dweight, p.dweight_partials,
                                    n.dx ? nullptr : side, sms, gave_up, stream);
        if (e == cudaSuccess && d_dweight && rows == 0)
            e = osr::launch_linear_zero(w.to, g_rows, g_cols, sms, stream);
    }
    return e == cudaSuccess ? ADAMW_OK : cuda_fail(cudaError_t(e), "linear layer launch");
}

}  // extern "C"
