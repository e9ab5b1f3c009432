// layernorm_bwd.cu -- joins the column sums of the layer norm's backward
// pass, and dispatches it by element type.
#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "early_dev.cuh"
#include "layernorm.h"

namespace osr {

template <typename T>
int launch_ln_backward_typed(const LnBackward& a, int sm_count, std::atomic<int>* known,
                             int32_t* parts, cudaStream_t s);

namespace {

constexpr int kCols = 32, kSlices = 32;  // of a block

// Adds the blocks' partial sums up, column by column: slice q of a block
// takes partials q, q + 32, ..., then the slices are added in order; blockIdx.y
// 0: dweight, 1: dbias.
__global__ void __launch_bounds__(kCols * kSlices) k_ln_grads(LnGrads g)
{
    detail::wait_before();
    detail::go_ahead();
    __shared__ float sums[kSlices][kCols];
    const int lane = threadIdx.x % kCols, slice = threadIdx.x / kCols;
    const int c = blockIdx.x * kCols + lane;
    void* const out = blockIdx.y ? g.dbias : g.dweight;
    if (!out)
        return;
    float s = 0.0f;
    if (c < g.cols) {
        const float* p = g.partials + int64_t(blockIdx.y) * g.cols + c;
#pragma unroll 4
        for (int q = slice; q < g.parts; q += kSlices)
            s += __ldcg(p + int64_t(q) * 2 * g.cols);
    }
    sums[slice][lane] = s;
    __syncthreads();
    if (slice || c >= g.cols)
        return;
#pragma unroll
    for (int q = 1; q < kSlices; ++q)
        s += sums[q][lane];
    if (g.dtype == kDtypeF32) {
        float* o = static_cast<float*>(out) + c;
        *o = g.accumulate ? *o + s : s;
    } else if (g.dtype == kDtypeBF16) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + c;
        *o = __float2bfloat16_rn(g.accumulate ? __bfloat162float(*o) + s : s);
    } else {
        __half* o = static_cast<__half*>(out) + c;
        *o = __float2half_rn(g.accumulate ? __half2float(*o) + s : s);
    }
}

}  // namespace

int launch_ln_backward(const LnBackward& a, int32_t dtype, int sm_count, LnBlocks& known,
                       int32_t* parts, void* stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == kDtypeBF16)
        return launch_ln_backward_typed<__nv_bfloat16>(a, sm_count, known.per_sm[dtype], parts, s);
    if (dtype == kDtypeF16)
        return launch_ln_backward_typed<__half>(a, sm_count, known.per_sm[dtype], parts, s);
    return launch_ln_backward_typed<float>(a, sm_count, known.per_sm[dtype], parts, s);
}

int launch_ln_grads(const LnGrads& g, void* stream)
{
    return detail::launch_early(&k_ln_grads, dim3(unsigned(detail::ceil_div(g.cols, kCols)), 2),
                                kCols * kSlices, 0, static_cast<cudaStream_t>(stream), g);
}

}  // namespace osr
