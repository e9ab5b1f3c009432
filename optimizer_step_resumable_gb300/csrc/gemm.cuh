// gemm.cuh -- C = A B^T on the fifth-generation tensor cores, with an epilogue
// of the caller's: out of each tile's float32 sums it makes whatever the
// operator stores.
//
// What bounds it: 2 m n k operations at the tensor cores' rate, as soon as
// tiles are read once from L2 for 256 x BN products each.  Two blocks of a
// cluster share a tile of 256 x BN: each holds half of A's rows and half of
// B's, so each reads half as much of B as it would alone.  A block's warps:
//   0      keeps a ring of tiles of 64 of the inner dimension full (bulk
//          tensor copies; the ring is as long as shared memory allows)
//   1      of the pair's first block: issues the products (one thread)
//   2      tensor memory
//   4..11  epilogue: warp w has the rows 32 (w % 4).. of the block's half of
//          the tile, and one half of the columns
// Sums take two halves of the tensor memory in turn, so that the epilogue of
// one tile runs beside the products of the next.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"
#include "early_dev.cuh"
#include "gemm.h"
#include "tensor_dev.cuh"

namespace osr {
namespace detail {

constexpr int kGemmThreads = 384;
constexpr int kGemmEpilogueWarps = 8;

template <int BN>
struct GemmRing {
    static constexpr int kRowsB = BN / 2;  // of B's tile, in a block
    // across, B comes in whole 64 rows
    static constexpr int kWholeB = kRowsB < 64 ? kRowsB : (kRowsB + 63) / 64 * 64;
    static constexpr int kBytesA = 128 * kGemmInner * 2, kBytesB = kWholeB * kGemmInner * 2;
    static constexpr int kStage = kBytesA + kBytesB;
    static constexpr int kStages = (192 * 1024) / kStage;
    static constexpr int kAccColumns = BN > 128 ? 256 : BN;  // of tensor memory, a tile
    static constexpr int kColumns = 2 * kAccColumns;  // a power of two from 32 to 512
    // tiles start on 1024 bytes; each warp of the epilogue has 32 x 33 floats
    static constexpr int kWarpStage = 32 * 33 * 4;
    static constexpr int kSmem = kStages * kStage + 1024 + kGemmEpilogueWarps * kWarpStage;
};

struct GemmItem {
    int32_t m0, tile_n, split, chain, first, last;  // rows, tile of columns, inner blocks
};

// Items in bands of 8 tiles of rows: the tiles that run at a time form a
// rectangle, whose rows and columns of A and B stay in L2.
__device__ __forceinline__ GemmItem gemm_item(const GemmShape& s, int32_t item, int32_t chain)
{
    const int32_t tiles = s.tiles_m * s.tiles_n;
    GemmItem it;
    it.split = item / tiles;
    const int32_t t = item - it.split * tiles;
    const int32_t band = t / (8 * s.tiles_n), r = t - band * 8 * s.tiles_n;
    const int32_t high = min(8, s.tiles_m - 8 * band);
    it.tile_n = r / high;
    it.m0 = (8 * band + r - it.tile_n * high) * kGemmTileM;
    it.chain = chain;
    const int64_t parts = int64_t(s.splits) * s.chains, part = int64_t(it.split) * s.chains + chain;
    it.first = int32_t(s.blocks * part / parts);
    it.last = int32_t(s.blocks * (part + 1) / parts);
    return it;
}
// The next item of a pair: its chains one after another, then `pairs` further.
__device__ __forceinline__ void gemm_next(const GemmShape& s, int32_t pairs, int32_t& item,
                                          int32_t& chain)
{
    if (++chain == s.chains) {
        chain = 0;
        item += pairs;
    }
}

// E: the epilogue.  E::Params is its arguments; an object of E is made for
// each tile and thread by E(params, shape, row, first column, columns, item,
// which half of the tile's columns, 32 x 33 floats of shared memory of the warp's own), gets the
// sums of its row by chunk(params, shape, column, number of the chunk, values,
// those floats) and ends with end(params, shape).
template <int BN, typename E>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    k_gemm(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
           const __grid_constant__ GemmShape s, const __grid_constant__ typename E::Params e)
{
    using R = GemmRing<BN>;
    extern __shared__ unsigned char raw[];
    __shared__ alignas(8) uint64_t bars[2 * R::kStages + 4];
    __shared__ uint32_t tmem_slot;
    __shared__ int gave_up;
    volatile int* const dead = &gave_up;

    const uint32_t warp = threadIdx.x / 32, rank = cluster_rank();
    const uint32_t ring = (smem_address(raw) + 1023) & ~1023u;
    const uint32_t full = smem_address(bars), empty = full + 8 * R::kStages;
    const uint32_t sums_full = empty + 8 * R::kStages, sums_empty = sums_full + 16;

    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int i = 0; i < R::kStages; ++i) {
            barrier_init(full + 8 * i, 1);
            barrier_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            barrier_init(sums_full + 8 * i, 1);
            barrier_init(sums_empty + 8 * i, 2 * kGemmEpilogueWarps);
        }
        barriers_visible();
        prefetch_map(&map_a);
        prefetch_map(&map_b);
    }
    __syncthreads();
    cluster_sync();
    if (warp == 2)
        tmem_alloc(smem_address(&tmem_slot), R::kColumns);
    before_sync();
    __syncthreads();
    after_sync();
    const uint32_t tmem = tmem_slot;
    wait_before();
    go_ahead();

    const int32_t items = s.tiles_m * s.tiles_n * s.splits;
    const int32_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;

    if (warp == 0 && elect_one()) {
        uint32_t stage = 0, phase = 0;
        const uint32_t full_first = in_block(full, 0);
        // of both blocks' tiles
        const uint32_t bytes =
            2 * (R::kBytesA + (s.b_across ? R::kBytesB : R::kRowsB * kGemmInner * 2));
        bool ok = true;
        for (int32_t item = pair, chain = 0; item < items && ok; gemm_next(s, pairs, item, chain)) {
            const GemmItem it = gemm_item(s, item, chain);
            const int32_t row_a = it.m0 + 128 * int32_t(rank);
            const int32_t row_b = it.tile_n * BN + R::kRowsB * int32_t(rank);
            for (int32_t k = it.first; k < it.last; ++k) {
                ok = barrier_wait(empty + 8 * stage, phase ^ 1, dead);
                if (!ok)
                    break;
                if (rank == 0)
                    barrier_expect(full + 8 * stage, bytes);
                const uint32_t bar = full_first + 8 * stage;
                const uint32_t to = ring + stage * R::kStage;
                const int32_t inner = k * kGemmInner;
                if (!s.a_across) {
                    load_tile(to, &map_a, inner, row_a, bar);
                } else {
                    load_tile(to, &map_a, row_a, inner, bar);
                    load_tile(to + 8192, &map_a, row_a + 64, inner, bar);
                }
                if (!s.b_across) {
                    load_tile(to + R::kBytesA, &map_b, inner, row_b, bar);
                } else {
#pragma unroll
                    for (int i = 0; i < R::kRowsB; i += 64)
                        load_tile(to + R::kBytesA + i * 128, &map_b, row_b + i, inner, bar);
                }
                if (++stage == R::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        // the pair's products still read what this block's last tiles hold, and
        // say so at its barriers: the block outlives that
        for (int i = 0; i < R::kStages && ok; ++i) {
            ok = barrier_wait(empty + 8 * stage, phase ^ 1, dead);
            if (++stage == R::kStages) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (!ok) {  // copies in flight land within microseconds
            const uint64_t begin = nanoseconds();
            while (nanoseconds() - begin < 5000000)
                ;
        }
    } else if (warp == 1 && rank == 0 && elect_one()) {
        uint32_t stage = 0, phase = 0;
        const uint32_t step_a = s.a_across ? 2048 : 32, step_b = s.b_across ? 2048 : 32;
        int32_t n = 0;
        bool ok = true;
        for (int32_t item = pair, chain = 0; item < items && ok;
             gemm_next(s, pairs, item, chain), ++n) {
            const GemmItem it = gemm_item(s, item, chain);
            const int32_t slot = n & 1;
            ok = barrier_wait(sums_empty + 8 * slot, ((n >> 1) & 1) ^ 1, dead);
            if (!ok)
                break;
            after_sync();
            const uint32_t d = tmem + uint32_t(slot * R::kAccColumns);
            for (int32_t k = it.first; k < it.last; ++k) {
                ok = barrier_wait(full + 8 * stage, phase, dead);
                if (!ok)
                    break;
                after_sync();
                const uint32_t at = ring + stage * R::kStage;
                const uint64_t a = tile_descriptor(at, 8192);
                const uint64_t b = tile_descriptor(at + R::kBytesA, 8192);
#pragma unroll
                for (int i = 0; i < kGemmInner / 16; ++i)
                    mma_pair(d, a + ((i * step_a) >> 4), b + ((i * step_b) >> 4), s.what,
                             k > it.first || i > 0);
                commit_pair(empty + 8 * stage);
                if (++stage == R::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (ok)
                commit_pair(sums_full + 8 * slot);
        }
    } else if (warp >= 4) {
        constexpr int kHalf = BN / 2, kChunk = kHalf < 32 ? kHalf : 32;
        const uint32_t quarter = warp % 4, half = (warp - 4) / 4;
        const uint32_t done = in_block(sums_empty, 0);
        float* const stage = reinterpret_cast<float*>(
            raw + (ring - smem_address(raw)) + R::kStages * R::kStage + (warp - 4) * R::kWarpStage);
        int32_t n = 0;
        for (int32_t item = pair, chain = 0; item < items; gemm_next(s, pairs, item, chain), ++n) {
            const GemmItem it = gemm_item(s, item, chain);
            const int32_t slot = n & 1;
            const int32_t row = it.m0 + 128 * int32_t(rank) + 32 * int32_t(quarter) +
                                int32_t(threadIdx.x % 32);
            const int32_t column = it.tile_n * BN + kHalf * int32_t(half);
            E epilogue(e, s, row, column, kHalf, it, int32_t(half), stage);
            const bool ok = barrier_wait(sums_full + 8 * slot, (n >> 1) & 1, dead);
            if (!__all_sync(0xFFFFFFFFu, ok))
                break;
            after_sync();
            const uint32_t from = tmem + uint32_t(slot * R::kAccColumns) + half * kHalf +
                                  ((32 * quarter) << 16);
#pragma unroll
            for (int c = 0; c < kHalf / kChunk; ++c) {
                float v[kChunk];
                __syncwarp();
                tmem_read(from + c * kChunk, v);
                tmem_wait(v);
                if (c + 1 == kHalf / kChunk) {  // all of this thread's sums are in registers
                    before_sync();
                    __syncwarp();
                    if (threadIdx.x % 32 == 0)
                        barrier_arrive_at(done + 8 * slot);
                }
                epilogue.chunk(e, s, column + c * kChunk, c, v, stage);
            }
            epilogue.end(e, s);
            __syncwarp();
        }
    }
    __syncwarp();
    before_sync();
    __syncthreads();
    cluster_sync();
    after_sync();
    if (warp == 2)
        tmem_free(tmem, R::kColumns);
    if (threadIdx.x == 0 && *dead && s.gave_up)
        *static_cast<volatile int32_t*>(s.gave_up) = 1;
}

// Launches it on as many pairs of blocks as there are items, or pairs of SMs.
template <int BN, typename E>
inline int gemm_launch(const CUtensorMap& a, const CUtensorMap& b, const GemmShape& s,
                       const typename E::Params& e, int sm_count, cudaStream_t stream)
{
    using R = GemmRing<BN>;
    const int64_t items = int64_t(s.tiles_m) * s.tiles_n * s.splits;
    const int pairs = int(items < sm_count / 2 ? items : sm_count / 2);
    const cudaError_t err = cudaFuncSetAttribute(
        k_gemm<BN, E>, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kSmem);
    if (err != cudaSuccess)
        return int(err);
    return launch_early(k_gemm<BN, E>, dim3(unsigned(2 * pairs)), kGemmThreads, R::kSmem, stream, a,
                        b, s, e);
}

}  // namespace detail
}  // namespace osr
