// layernorm.h -- the layer norm: what its entry points (layernorm_api.cu) and
// its kernels share.  Not part of the ABI.
#pragma once

#include <atomic>
#include <cstdint>

#include "internal.h"

namespace osr {

struct LnForward {
    const void* x;
    int64_t x_stride;
    const void* weight;  // NULL: 1
    const void* bias;    // NULL: 0
    void* y;
    int64_t y_stride;
    float* mean;  // NULL: not kept
    float* rstd;
    int64_t rows;
    int32_t cols;
    float eps;
    bool w_f32;  // weight and bias are float32, not the type of x
};

struct LnBackward {
    const void* dy;
    int64_t dy_stride;
    const void* x;
    int64_t x_stride;
    const void* weight;  // NULL: 1
    const float* mean;
    const float* rstd;
    void* dx;
    int64_t dx_stride;
    int64_t rows;
    int32_t cols;
    bool w_f32;
    bool sums;        // dweight or dbias is wanted
    float* partials;  // per block: cols sums of dy xhat, then cols of dy
};

// What the second kernel of the backward pass joins.
struct LnGrads {
    const float* partials;
    int32_t parts;  // blocks that wrote partials
    int32_t cols;
    void* dweight;
    void* dbias;
    int32_t dtype;
    bool accumulate;
};

// Rows wider than this do not fit the registers of one block.
constexpr int kLnRegisterCols = 16384;
// Blocks of the backward pass that write partial sums, at most.
inline int ln_parts_max(int32_t cols) { return cols <= 4096 ? 608 : 304; }
constexpr int kLnWideParts = 32;  // strips of rows, for rows wider than the registers

// Number of partial sums a context needs room for.
inline int64_t ln_partials(int32_t cols)
{
    const int parts = cols > kLnRegisterCols ? kLnWideParts : ln_parts_max(cols);
    return int64_t(parts) * 2 * cols;
}

// Resident blocks per SM of the kernels of one pass, on the context's device
// and for its cols, which leave one kernel for each element type and way the
// rows lie (layernorm_dev.cuh); 0: not asked for yet, so the kernel may not
// have been allowed its shared memory on this device either.
constexpr int kLnDtypes = 3, kLnRows = 5;
struct LnBlocks {
    std::atomic<int> per_sm[kLnDtypes][kLnRows] = {};
};

int launch_ln_forward(const LnForward& a, int32_t dtype, int sm_count, LnBlocks& known,
                      void* stream);
// Writes dx and, if a.sums, *parts partial sums.
int launch_ln_backward(const LnBackward& a, int32_t dtype, int sm_count, LnBlocks& known,
                       int32_t* parts, void* stream);
int launch_ln_grads(const LnGrads& g, void* stream);

}  // namespace osr
