// gemm.h -- the tiled matrix product on the tensor cores that the linear
// layer and the cross entropy share: what the host code that plans and
// launches it needs.  Not part of the ABI.
#pragma once

#include <cstdint>

#include <cuda.h>

#include "internal.h"

namespace osr {

// A matrix of 16-bit elements as an operand.  `outer` is the dimension that
// appears in the product, `inner` the one that is summed over.  `across`:
// elements that are adjacent in memory are neighbours in the outer dimension.
struct GemmOperand {
    const void* p;
    int64_t outer, inner;
    int64_t stride;  // elements between two rows of memory
    bool across;
};

// What the kernel is told about one product of `m` x `n` over the inner
// dimension, in tiles of 256 x BN shared by two blocks, the inner dimension
// cut into `splits` ranges of blocks of 64, and each of those into `chains`
// that one pair of blocks sums up one after another: the tensor cores cut
// their sums, so long ones lose bits.
struct GemmShape {
    int32_t m, n;
    int32_t tiles_m, tiles_n, splits, chains, blocks;
    uint32_t what;  // mma_what
    int32_t a_across, b_across;
    int32_t* gave_up;  // set to 1 if a wait ran out (host memory)
};

// How the items of two products are dealt out to the pairs of blocks, the long
// items first: pair p gets every `pairs`-th of the `longs`, then, of the
// `shorts`, `after` if it has one long more than others (p < ahead), else
// `before`.
struct GemmDeal {
    int32_t pairs, longs, ahead, shorts, after, before;
};

// Sums of columns over `strips` rows of float32, in order, written to or (add)
// added to out.
struct GemmSide {
    const float* partials;  // NULL: nothing to do
    int32_t strips;
    int64_t columns;
    void* out;
    int32_t dtype;
    bool add;
};

constexpr int kGemmTileM = 256, kGemmInner = 64;

// Whether the tiled copies can read a matrix: its address and row distance on
// 16-byte boundaries.
inline bool gemm_readable(const void* p, int64_t stride)
{
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0;
}

// Resolves the driver's encoder of tensor maps, once a process; cudaError_t.
int gemm_init();
// The map of an operand whose tile in a block is `rows` x 64 of the outer and
// the inner dimension.
int gemm_map(const GemmOperand& o, int rows, bool bf16, CUtensorMap* map);

}  // namespace osr
