// distill.h -- the distillation from a teacher's top logits: what its entry
// points (distill_api.cu) and its kernels share.  Not part of the ABI.
#pragma once

#include <cstdint>

#include "internal.h"

namespace osr {

constexpr int32_t kDistillMost = 1024;  // entries of a teacher's row

struct Distill {
    const void* logits;
    int64_t stride;
    int32_t dtype;
    int32_t vocab;
    const int64_t* ids;  // rows x k; below 0: no entry
    const void* values;  // rows x k
    int32_t values_dtype;
    int32_t k;
    float temperature;
    int64_t rows;
    float* loss;          // forward
    float* lse;           // forward; NULL: not kept
    const float* lse_in;  // backward
    const float* dloss;   // NULL: 1
    float scale;
    void* dlogits;  // may be logits
    int64_t dlogits_stride;
};

int launch_distill_forward(const Distill& a, void* stream);
int launch_distill_backward(const Distill& a, void* stream);

}  // namespace osr
