// distill_api.cu -- the C ABI entry points of the distillation from a
// teacher's top logits (distill_* of include/adamw_ckpt.h).
#include <cmath>
#include <cstdint>
#include <new>

#include <cuda_runtime.h>

#include "api_util.h"
#include "arrays.h"
#include "distill.h"

struct distill_ctx {
    int device = -1;
    int32_t vocab = 0, k = 0;
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

constexpr int32_t kMaxVocab = 1 << 30;

int check_common(const distill_ctx* ctx, const void* d_logits, int64_t stride, int32_t dtype,
                 const int64_t* d_ids, const void* d_values, int32_t values_dtype,
                 double temperature, int64_t rows)
{
    if (!ctx)
        return fail(ADAMW_EINVAL, "ctx is NULL");
    if (!known_dtype(dtype))
        return fail(ADAMW_EINVAL, "dtype=%d is not F32, BF16 or F16", dtype);
    if (!known_dtype(values_dtype))
        return fail(ADAMW_EINVAL, "values_dtype=%d is not F32, BF16 or F16", values_dtype);
    if (rows < 0 || rows > INT32_MAX)
        return fail(ADAMW_EINVAL, "rows=%lld outside [0, 2^31 - 1]", (long long)rows);
    // beyond, T^2 or log2(e) / T leaves float32: the loss would be 0, infinity or NaN
    if (!(temperature >= std::ldexp(1.0, -60) && temperature <= std::ldexp(1.0, 60)))
        return fail(ADAMW_EINVAL, "temperature=%g outside [2^-60, 2^60]", temperature);
    int rc;
    if ((rc = check_rows(d_logits, stride, rows, ctx->vocab, size_of(dtype), "d_logits")) ||
        (rc = check_array(d_ids, 8, rows == 0, "d_ids")) ||
        (rc = check_array(d_values, size_of(values_dtype), rows == 0, "d_values")))
        return rc;
    return ADAMW_OK;
}

osr::Distill arguments(const distill_ctx* ctx, const void* d_logits, int64_t stride, int32_t dtype,
                       const int64_t* d_ids, const void* d_values, int32_t values_dtype,
                       double temperature, int64_t rows)
{
    osr::Distill a{};
    a.logits = d_logits;
    a.stride = stride;
    a.dtype = dtype;
    a.vocab = ctx->vocab;
    a.ids = d_ids;
    a.values = d_values;
    a.values_dtype = values_dtype;
    a.k = ctx->k;
    a.temperature = float(temperature);
    a.rows = rows;
    return a;
}

}  // namespace

extern "C" {

int distill_create(int32_t vocab, int32_t k, distill_ctx** out)
{
    osr::clear_error();
    if (!out)
        return fail(ADAMW_EINVAL, "out is NULL");
    *out = nullptr;
    if (vocab < 1 || vocab > kMaxVocab)
        return fail(ADAMW_EINVAL, "vocab=%d outside [1, 2^30]", vocab);
    if (k < 1 || k > osr::kDistillMost)
        return fail(ADAMW_EINVAL, "k=%d outside [1, %d]", k, osr::kDistillMost);
    distill_ctx* c = new (std::nothrow) distill_ctx;
    if (!c)
        return fail(ADAMW_EINVAL, "out of host memory");
    c->vocab = vocab;
    c->k = k;
    const cudaError_t e = cudaGetDevice(&c->device);
    if (e != cudaSuccess) {
        delete c;
        return cuda_fail(e, "cudaGetDevice");
    }
    *out = c;
    return ADAMW_OK;
}

int distill_destroy(distill_ctx* ctx)
{
    osr::clear_error();
    delete ctx;
    return ADAMW_OK;
}

int distill_forward(distill_ctx* ctx, const void* d_logits, int64_t logits_stride, int32_t dtype,
                    const int64_t* d_ids, const void* d_values, int32_t values_dtype,
                    double temperature, float* d_loss, float* d_lse, int64_t rows, void* stream)
{
    osr::clear_error();
    int rc = check_common(ctx, d_logits, logits_stride, dtype, d_ids, d_values, values_dtype,
                          temperature, rows);
    if (rc != ADAMW_OK)
        return rc;
    if ((rc = check_array(d_loss, 4, rows == 0, "d_loss")) ||
        (rc = check_array(d_lse, 4, true, "d_lse")))
        return rc;
    const int64_t entries = rows * ctx->k;
    const Pieces outs[] = {vector_of(d_loss, rows, 4, "d_loss"),
                           vector_of(d_lse, rows, 4, "d_lse")};
    const Pieces ins[] = {rows_of(d_logits, logits_stride, rows, ctx->vocab, size_of(dtype),
                                  "d_logits"),
                          vector_of(d_ids, entries, 8, "d_ids"),
                          vector_of(d_values, entries, size_of(values_dtype), "d_values")};
    if ((rc = check_apart(outs, ins)))
        return rc;
    if (rows == 0)
        return ADAMW_OK;
    DeviceScope scope(ctx->device);
    osr::Distill a = arguments(ctx, d_logits, logits_stride, dtype, d_ids, d_values, values_dtype,
                               temperature, rows);
    a.loss = d_loss;
    a.lse = d_lse;
    const int e = osr::launch_distill_forward(a, stream);
    return e == cudaSuccess ? ADAMW_OK : cuda_fail(cudaError_t(e), "distillation launch");
}

int distill_backward(distill_ctx* ctx, const void* d_logits, int64_t logits_stride, int32_t dtype,
                     const int64_t* d_ids, const void* d_values, int32_t values_dtype,
                     double temperature, const float* d_lse, const float* d_dloss, double scale,
                     void* d_dlogits, int64_t dlogits_stride, int64_t rows, void* stream)
{
    osr::clear_error();
    int rc = check_common(ctx, d_logits, logits_stride, dtype, d_ids, d_values, values_dtype,
                          temperature, rows);
    if (rc != ADAMW_OK)
        return rc;
    const size_t s = size_of(dtype);
    if ((rc = check_array(d_lse, 4, rows == 0, "d_lse")) ||
        (rc = check_array(d_dloss, 4, true, "d_dloss")) ||
        (rc = check_rows(d_dlogits, dlogits_stride, rows, ctx->vocab, s, "d_dlogits")))
        return rc;
    if (!std::isfinite(float(scale)))
        return fail(ADAMW_EINVAL, "scale=%g is not finite", scale);
    const bool in_place = d_dlogits == d_logits && (dlogits_stride == logits_stride || rows <= 1);
    const int64_t entries = rows * ctx->k;
    const Pieces outs[] = {rows_of(d_dlogits, dlogits_stride, rows, ctx->vocab, s, "d_dlogits")};
    const Pieces ins[] = {rows_of(d_logits, logits_stride, in_place ? 0 : rows, ctx->vocab, s,
                                  "d_logits"),
                          vector_of(d_ids, entries, 8, "d_ids"),
                          vector_of(d_values, entries, size_of(values_dtype), "d_values"),
                          vector_of(d_lse, rows, 4, "d_lse"),
                          vector_of(d_dloss, rows, 4, "d_dloss")};
    if ((rc = check_apart(outs, ins)))
        return rc;
    if (rows == 0)
        return ADAMW_OK;
    DeviceScope scope(ctx->device);
    osr::Distill a = arguments(ctx, d_logits, logits_stride, dtype, d_ids, d_values, values_dtype,
                               temperature, rows);
    a.lse_in = d_lse;
    a.dloss = d_dloss;
    a.scale = float(scale);
    a.dlogits = d_dlogits;
    a.dlogits_stride = dlogits_stride;
    const int e = osr::launch_distill_backward(a, stream);
    return e == cudaSuccess ? ADAMW_OK : cuda_fail(cudaError_t(e), "distillation launch");
}

}  // extern "C"
