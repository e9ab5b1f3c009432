// linear.h -- the linear layer: what its entry points (linear_api.cu) and its
// kernels share.  Not part of the ABI.
#pragma once

#include <cstdint>

#include "gemm.h"
#include "internal.h"

namespace osr {

// Where a product goes: out = act(alpha sum + bias) + residual, which may be
// out itself: added to what is there.  The row distances are in elements.
struct LinearOut {
    void* out;
    int64_t stride;
    int32_t dtype;  // of out and z
    const void* bias;  // NULL: 0; one per column
    int32_t bias_dtype;
    const void* residual;  // NULL: none; may be out
    int64_t residual_stride;
    int32_t residual_dtype;
    void* z;  // NULL: not kept
    int64_t z_stride;
    int32_t act;
    float alpha;
    const float* alpha_factor;  // on the device, multiplies alpha; NULL: 1
    int32_t vectors;            // rows of out, residual and z on 32-byte boundaries
};

// out (rows x columns) from a (rows x inner) and b (columns x inner).
struct LinearProduct {
    GemmOperand a, b;
    bool bf16;
    LinearOut to;
};
// Makes a product add to what is there.
inline void accumulate_into(LinearOut& o)
{
    o.residual = o.out;
    o.residual_stride = o.stride;
    o.residual_dtype = o.dtype;
}

// How it is computed: in tiles of 256 x bn with the inner dimension in
// `splits` ranges, each in `chains` (see GemmShape), and the sums joined by a
// second kernel if there are `partials`; swapped: the tile's long side lies along
// the columns, for products of few rows.
struct LinearPlan {
    bool few;  // not in tiles at all (linear_few.cu)
    bool swapped;
    int32_t bn, splits, chains;
    int64_t partials;  // float32 sums in the workspace; 0: they go out as they are
};
// How many blocks of the inner dimension (kGemmInner products each) the tensor
// cores may sum in one go for an output of the type.  They cut instead of rounding:
// a sum of equal signs loses 1.7 x 2^-24 of itself for each 16 products of binary16
// (measured from 4096 to 32768 products; of bfloat16, whose products have fewer bits,
// 0.8 to 1.5).  So 2^14 products lose 1.0e-4, 0.21 of binary16's rounding, 2^17
// at most 8.3e-4, 0.21 of bfloat16's, and 1024 at most 6.5e-6.
inline int64_t linear_chain(int32_t dtype)
{
    return dtype == ADAMW_DTYPE_F32 ? 16 : dtype == ADAMW_DTYPE_BF16 ? 2048 : 256;
}
// Whether a sum over one of these may need chains for a 16-bit output.
inline bool linear_long(int64_t a, int64_t b, int64_t c)
{
    const int64_t most = linear_chain(ADAMW_DTYPE_F16) * kGemmInner;
    return a > most || b > most || c > most;
}
// *_across: whether the operand's outer dimension is the adjacent one; f32: out
// is float32; chain: linear_chain of the type that the sum is rounded to in the end.
struct LinearSize {
    int64_t rows, columns, inner;
    bool a_across, b_across, f32;
    int64_t chain;
};
LinearPlan linear_plan(const LinearSize& p, int sm_count);
// Plans of two products that do not depend on one another; true if they go in
// one launch.
bool linear_plan_two(const LinearSize& p, const LinearSize& q, int sm_count, LinearPlan* p_plan,
                     LinearPlan* q_plan);
// About how many microseconds one or two (q not NULL) products take in whole
// tiles of 256 x 256.
double linear_us(const LinearSize& p, const LinearSize* q, int sm_count);
// side (may be NULL): done in the same launch, by a warp that has nothing else
// to do, or in one of its own.
int linear_product(const LinearProduct& p, const LinearPlan& plan, float* partials,
                   const GemmSide* side, int sm_count, int32_t* gave_up, void* stream);
// Two plain products (neither bias nor activation nor z) in one launch.
int linear_product_two(const LinearProduct& p, const LinearPlan& p_plan, float* p_partials,
                       const LinearProduct& q, const LinearPlan& q_plan, float* q_partials,
                       const GemmSide* side, int sm_count, int32_t* gave_up, void* stream);
// A product of few rows that lie along the sum, and whether that is faster.
bool linear_few_pays(const LinearSize& p);
int linear_few(const LinearProduct& p, int sm_count, void* stream);
// A product over nothing.
int launch_linear_zero(const LinearOut& to, int64_t rows, int64_t columns, int sm_count,
                       void* stream);

// Rows of 16-bit elements, copied to where the tiled copies can read them;
// `to` NULL: none.
struct LinearCopy {
    const void* from;
    int64_t from_stride;
    void* to;
    int64_t to_stride, rows, columns;
};
int launch_linear_copies(const LinearCopy& a, const LinearCopy& b, void* stream);

// dz = dy act'(z), rounded to their type, into rows of `stride` elements, and
// its column sums (of the unrounded values) in strips; two copies beside it.
struct LinearSlope {
    const void* dy;
    int64_t dy_stride;
    const void* z;  // NULL if act is LINEAR_NONE
    int64_t z_stride;
    int32_t act;
    bool bf16;
    void* dz;  // NULL: not wanted
    int64_t stride;
    int64_t rows, columns;
    float* partials;  // strips x columns; NULL: no sums
    int32_t strips;
    LinearCopy copies[2];
};
int linear_strips(int64_t rows, int64_t columns, int sm_count);
int launch_linear_slope(const LinearSlope& a, void* stream);
// The strips' sums joined, in a launch of its own.
int launch_linear_bias_grad(const GemmSide& side, void* stream);

}  // namespace osr
