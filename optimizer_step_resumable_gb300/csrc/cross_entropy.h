// cross_entropy.h -- the cross entropy over a vocabulary whose logits are not
// kept: what its entry points (cross_entropy_api.cu) and its kernels share.
// Not part of the ABI.
#pragma once

#include <cstdint>

#include "gemm.h"
#include "internal.h"

namespace osr {

// Columns of logits in a tile, and the parts of it that a row's threads of
// the epilogue have.
constexpr int kCeColumns = 256, kCeParts = 2;

// Forward, first kernel: for each row and each half of a tile of columns the
// largest logit and the sum of exponentials relative to it, in powers of two,
// and the target's logit.
struct CeForward {
    GemmOperand x, weight;
    bool bf16;
    const int64_t* target;
    float2* parts;  // parts x rows
    float* at;      // the target's logit, one a row
};
int launch_ce_parts(const CeForward& a, int sm_count, int32_t* gave_up, void* stream);
// Second kernel: joins them.
struct CeJoin {
    const float2* parts;
    int32_t count;
    const float* at;
    const int64_t* target;
    int64_t rows;
    int32_t vocab;
    float z_loss;
    float* loss;
    float* lse;  // NULL: not kept
};
int launch_ce_join(const CeJoin& a, void* stream);

// What the gradient of the rows' logits is made of besides them.
struct CeFactors {
    const int64_t* target;
    const float* lse;
    const float* dloss;  // NULL: 1
    float two_z;  // twice z_loss
    int32_t vocab;
    const float* norm;  // multiplies the factors, on the device; NULL: 1
};
// For binary16: norms[0], a power of two that keeps the gradients in its range,
// and norms[1], which undoes it.
int launch_ce_norm(const CeFactors& f, int64_t rows, float* norms, void* stream);

// The gradient of the logits of a piece of the vocabulary: rows of `stride`
// 16-bit elements, a multiple of kCeColumns and at least the piece.
struct CeGradient {
    GemmOperand x, weight;  // the piece's rows of the weight
    bool bf16;
    CeFactors factors;
    int32_t first;  // the piece's place in the vocabulary
    void* gradient;
    int64_t stride;
};
int launch_ce_gradient(const CeGradient& a, int sm_count, int32_t* gave_up, void* stream);

}  // namespace osr
