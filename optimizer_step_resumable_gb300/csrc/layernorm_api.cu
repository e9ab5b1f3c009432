// layernorm_api.cu -- the C ABI entry points of the layer norm
// (layernorm_* of include/adamw_ckpt.h).
#include <cmath>
#include <cstdint>
#include <new>

#include <cuda_runtime.h>

#include "api_util.h"
#include "arrays.h"
#include "internal.h"
#include "layernorm.h"

struct layernorm_ctx {
    int device = -1;
    int sm_count = 0;
    int32_t cols = 0;
    float* d_partials = nullptr;
    osr::LnBlocks forward, backward;
};

namespace {

using osr::check_apart;
using osr::check_array;
using osr::check_rows;
using osr::cuda_fail;
using osr::DeviceScope;
using osr::fail;
using osr::known_dtype;
using osr::Pieces;
using osr::rows_of;
using osr::size_of;
using osr::vector_of;

constexpr int32_t kMaxCols = 1 << 18;

void free_ctx(layernorm_ctx* c)
{
    if (!c)
        return;
    if (c->device >= 0) {
        DeviceScope scope(c->device);
        if (c->d_partials) cudaFree(c->d_partials);  // waits for kernels that use it
    }
    delete c;
}

int create_ctx(layernorm_ctx* c)
{
    cudaError_t e = cudaGetDevice(&c->device);
    if (e != cudaSuccess) {
        c->device = -1;
        return cuda_fail(e, "cudaGetDevice");
    }
    CUDA_TRY(cudaDeviceGetAttribute(&c->sm_count, cudaDevAttrMultiProcessorCount, c->device));
    CUDA_TRY(cudaMalloc(&c->d_partials, sizeof(float) * size_t(osr::ln_partials(c->cols))));
    return ADAMW_OK;
}

int check_common(const layernorm_ctx* ctx, int32_t x_dtype, int32_t w_dtype, int64_t rows)
{
    if (!ctx)
        return fail(ADAMW_EINVAL, "ctx is NULL");
    if (!known_dtype(x_dtype))
        return fail(ADAMW_EINVAL, "x_dtype=%d is not F32, BF16 or F16", x_dtype);
    if (w_dtype != ADAMW_DTYPE_F32 && w_dtype != x_dtype)
        return fail(ADAMW_EINVAL, "w_dtype=%d is neither F32 nor x_dtype=%d", w_dtype, x_dtype);
    if (rows < 0)
        return fail(ADAMW_EINVAL, "rows=%lld is negative", (long long)rows);
    return ADAMW_OK;
}

}  // namespace

extern "C" {

int layernorm_create(int32_t cols, layernorm_ctx** out)
{
    osr::clear_error();
    if (!out)
        return fail(ADAMW_EINVAL, "out is NULL");
    *out = nullptr;
    if (cols < 1 || cols > kMaxCols)
        return fail(ADAMW_EINVAL, "cols=%d outside [1, 2^18]", cols);
    layernorm_ctx* c = new (std::nothrow) layernorm_ctx;
    if (!c)
        return fail(ADAMW_EINVAL, "out of host memory");
    c->cols = cols;
    const int rc = create_ctx(c);
    if (rc != ADAMW_OK) {
        free_ctx(c);
        return rc;
    }
    *out = c;
    return ADAMW_OK;
}

int layernorm_destroy(layernorm_ctx* ctx)
{
    osr::clear_error();
    free_ctx(ctx);
    return ADAMW_OK;
}

int layernorm_forward(layernorm_ctx* ctx, const void* d_x, int64_t x_stride, int32_t x_dtype,
                      const void* d_weight, const void* d_bias, int32_t w_dtype, void* d_y,
                      int64_t y_stride, float* d_mean, float* d_rstd, int64_t rows, double eps,
                      void* stream)
{
    osr::clear_error();
    int rc = check_common(ctx, x_dtype, w_dtype, rows);
    if (rc != ADAMW_OK)
        return rc;
    const size_t s = size_of(x_dtype), ws = size_of(w_dtype);
    if ((rc = check_rows(d_x, x_stride, rows, ctx->cols, s, "d_x")) ||
        (rc = check_rows(d_y, y_stride, rows, ctx->cols, s, "d_y")) ||
        (rc = check_array(d_weight, ws, true, "d_weight")) ||
        (rc = check_array(d_bias, ws, true, "d_bias")) ||
        (rc = check_array(d_mean, 4, true, "d_mean")) ||
        (rc = check_array(d_rstd, 4, true, "d_rstd")))
        return rc;
    if (!(eps >= 0.0 && std::isfinite(eps)))
        return fail(ADAMW_EINVAL, "eps=%g must be finite and >= 0", eps);
    const int64_t cols = ctx->cols;
    const Pieces out[] = {rows_of(d_y, y_stride, rows, cols, s, "d_y"),
                          vector_of(d_mean, rows, 4, "d_mean"),
                          vector_of(d_rstd, rows, 4, "d_rstd")};
    const Pieces in[] = {rows_of(d_x, x_stride, rows, cols, s, "d_x"),
                         vector_of(d_weight, cols, ws, "d_weight"),
                         vector_of(d_bias, cols, ws, "d_bias")};
    if ((rc = check_apart(out, in)))
        return rc;
    if (rows == 0)
        return ADAMW_OK;
    DeviceScope scope(ctx->device);
    const osr::LnForward a{d_x,    x_stride, d_weight, d_bias, d_y,        y_stride,
                           d_mean, d_rstd,   rows,     ctx->cols, float(eps),
                           w_dtype == ADAMW_DTYPE_F32};
    const int e = osr::launch_ln_forward(a, x_dtype, ctx->sm_count, ctx->forward, stream);
    return e == cudaSuccess ? ADAMW_OK : cuda_fail(cudaError_t(e), "layer norm launch");
}

int layernorm_backward(layernorm_ctx* ctx, const void* d_dy, int64_t dy_stride, const void* d_x,
                       int64_t x_stride, int32_t x_dtype, const void* d_weight, int32_t w_dtype,
                       const float* d_mean, const float* d_rstd, void* d_dx, int64_t dx_stride,
                       void* d_dweight, void* d_dbias, int32_t grad_dtype, int64_t rows,
                       int32_t flags, void* stream)
{
    osr::clear_error();
    int rc = check_common(ctx, x_dtype, w_dtype, rows);
    if (rc != ADAMW_OK)
        return rc;
    if (!known_dtype(grad_dtype))
        return fail(ADAMW_EINVAL, "grad_dtype=%d is not F32, BF16 or F16", grad_dtype);
    if (flags & ~LAYERNORM_ACCUMULATE)
        return fail(ADAMW_EINVAL, "unknown flags 0x%x", flags);
    const size_t s = size_of(x_dtype), gs = size_of(grad_dtype);
    if ((rc = check_rows(d_dy, dy_stride, rows, ctx->cols, s, "d_dy")) ||
        (rc = check_rows(d_x, x_stride, rows, ctx->cols, s, "d_x")) ||
        (rc = check_rows(d_dx, dx_stride, rows, ctx->cols, s, "d_dx")) ||
        (rc = check_array(d_weight, size_of(w_dtype), true, "d_weight")) ||
        (rc = check_array(d_mean, 4, rows == 0, "d_mean")) ||
        (rc = check_array(d_rstd, 4, rows == 0, "d_rstd")) ||
        (rc = check_array(d_dweight, gs, true, "d_dweight")) ||
        (rc = check_array(d_dbias, gs, true, "d_dbias")))
        return rc;
    const int64_t cols = ctx->cols;
    const Pieces out[] = {rows_of(d_dx, dx_stride, rows, cols, s, "d_dx"),
                          vector_of(d_dweight, cols, gs, "d_dweight"),
                          vector_of(d_dbias, cols, gs, "d_dbias")};
    const Pieces in[] = {rows_of(d_dy, dy_stride, rows, cols, s, "d_dy"),
                         rows_of(d_x, x_stride, rows, cols, s, "d_x"),
                         vector_of(d_weight, cols, size_of(w_dtype), "d_weight"),
                         vector_of(d_mean, rows, 4, "d_mean"),
                         vector_of(d_rstd, rows, 4, "d_rstd")};
    if ((rc = check_apart(out, in)))
        return rc;
    DeviceScope scope(ctx->device);
    const bool sums = d_dweight || d_dbias;
    int32_t parts = 0;
    int e = cudaSuccess;
    if (rows > 0) {
        const osr::LnBackward a{d_dy,   dy_stride, d_x,       x_stride, d_weight,
                                d_mean, d_rstd,    d_dx,      dx_stride, rows,
                                ctx->cols, w_dtype == ADAMW_DTYPE_F32, sums, ctx->d_partials};
        e = osr::launch_ln_backward(a, x_dtype, ctx->sm_count, ctx->backward, &parts, stream);
    }
    if (e == cudaSuccess && sums)
        e = osr::launch_ln_grads(osr::LnGrads{ctx->d_partials, parts, ctx->cols, d_dweight,
                                              d_dbias, grad_dtype,
                                              (flags & LAYERNORM_ACCUMULATE) != 0},
                                 stream);
    return e == cudaSuccess ? ADAMW_OK : cuda_fail(cudaError_t(e), "layer norm launch");
}

}  // extern "C"
