// layernorm_api.cu -- the C ABI entry points of the layer norm
// (layernorm_* of include/adamw_ckpt.h).
#include <cmath>
#include <cstdint>
#include <new>

#include <cuda_runtime.h>

#include "api_util.h"
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

using osr::cuda_fail;
using osr::DeviceScope;
using osr::fail;

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

bool known_dtype(int32_t d)
{
    return d == ADAMW_DTYPE_F32 || d == ADAMW_DTYPE_BF16 || d == ADAMW_DTYPE_F16;
}
size_t size_of(int32_t d) { return d == ADAMW_DTYPE_F32 ? 4 : 2; }

int check_array(const void* p, size_t size, bool optional, const char* name)
{
    if (!p && !optional)
        return fail(ADAMW_EINVAL, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % size)
        return fail(ADAMW_EINVAL, "%s is not %d-byte aligned", name, int(size));
    return ADAMW_OK;
}

int check_rows(const void* p, int64_t stride, int64_t rows, int32_t cols, size_t size,
               const char* name)
{
    if (const int rc = check_array(p, size, rows == 0, name))
        return rc;
    if (stride < cols && rows > 1)
        return fail(ADAMW_EINVAL, "%s: rows %lld apart, of %d elements", name, (long long)stride,
                    cols);
    return ADAMW_OK;
}

// `rows` pieces of `bytes` each, `stride` bytes apart (0 for a single one); a
// vector is one piece.
struct Pieces {
    uintptr_t begin;
    int64_t stride, rows, bytes;
    const char* name;
};
Pieces rows_of(const void* p, int64_t stride, int64_t rows, int64_t cols, size_t size,
               const char* name)
{
    return Pieces{reinterpret_cast<uintptr_t>(p), rows > 1 ? stride * int64_t(size) : 0, rows,
                  cols * int64_t(size), name};
}
Pieces vector_of(const void* p, int64_t n, size_t size, const char* name)
{
    return Pieces{reinterpret_cast<uintptr_t>(p), 0, p && n ? 1 : 0, n * int64_t(size), name};
}

// Whether a piece of `bytes` at `begin` shares a byte with some row of b.
bool touches(uintptr_t begin, int64_t bytes, const Pieces& b)
{
    // the last row that starts before the piece's end
    const int64_t before = int64_t(begin - b.begin) + bytes - 1;
    if (before < 0)
        return false;
    int64_t j = b.rows > 1 ? before / b.stride : 0;
    j = j < b.rows ? j : b.rows - 1;
    return j * b.stride + b.bytes > int64_t(begin - b.begin);
}
// Whether any byte belongs to both.  Rows of two arrays may lie between one
// another (columns of one matrix), so the ranges alone do not say.
bool overlap(const Pieces& a, const Pieces& b)
{
    if (a.rows == 0 || b.rows == 0)
        return false;
    const uintptr_t a_end = a.begin + uintptr_t((a.rows - 1) * a.stride + a.bytes);
    const uintptr_t b_end = b.begin + uintptr_t((b.rows - 1) * b.stride + b.bytes);
    if (a.begin >= b_end || b.begin >= a_end)
        return false;
    const Pieces &few = a.rows < b.rows ? a : b, &many = a.rows < b.rows ? b : a;
    // rows as far apart as the other's lie alike to it: the first that is
    // within the other's range, and the one before it, stand for all
    const bool alike = few.rows > 1 && few.stride == many.stride;
    int64_t i = 0, end = few.rows;
    if (alike) {
        const int64_t ahead = int64_t(many.begin - few.begin);
        i = ahead > 0 ? ahead / few.stride : 0;
        end = i + 2 < end ? i + 2 : end;
    }
    for (; i < end; ++i)
        if (touches(few.begin + uintptr_t(i * few.stride), few.bytes, many))
            return true;
    return false;
}
// Outputs share no byte with an input or with one another.
template <int kOut, int kIn>
int check_apart(const Pieces (&out)[kOut], const Pieces (&in)[kIn])
{
    for (int i = 0; i < kOut; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j]))
                return fail(ADAMW_EINVAL, "%s overlaps %s", out[i].name, out[j].name);
        for (int j = 0; j < kIn; ++j)
            if (overlap(out[i], in[j]))
                return fail(ADAMW_EINVAL, "%s overlaps %s", out[i].name, in[j].name);
    }
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
