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
//   3      sums that have to be joined meanwhile (GemmSide)
//   4..11  epilogue: warp w has the rows 32 (w % 4).. of the block's half of
//          the tile, and one half of the columns
// Sums take two halves of the tensor memory in turn, so that the epilogue of
// one tile runs beside the products of the next.
//
// An item is a tile or a part of one.  The items of one product take alike long
// and are dealt out in turn.  A launch may hold two products: what the one
// leaves idle at the end the other fills, and the start of a launch, some 5 us,
// is paid once.  The longer items are dealt out first, the others so that all
// pairs end together (GemmDeal).  (Items handed out by the hardware, by taking
// over clusters that have not started, cost about 1 us a tile.)
#pragma once

#include <type_traits>

#include <cuda_runtime.h>

#include "common.cuh"
#include "early_dev.cuh"
#include "gemm.h"
#include "linear_dev.cuh"
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

// The i-th item of pair p, or -1; those of the second product follow the
// first's.
__device__ __forceinline__ int32_t gemm_dealt(const GemmDeal& d, int32_t p, int32_t i)
{
    const int32_t longs = (d.longs - p + d.pairs - 1) / d.pairs;
    if (i < longs)
        return p + i * d.pairs;
    const int32_t j = i - longs;
    if (j >= (p < d.ahead ? d.after : d.before))
        return -1;
    const int32_t k = j < d.after ? j * d.pairs + p
                                  : d.after * d.pairs + (j - d.after) * (d.pairs - d.ahead) +
                                        (p - d.ahead);
    return k < d.shorts ? d.longs + k : -1;
}

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

// Warp `w` of `count`: 32 columns at a time.
__device__ __forceinline__ void gemm_side(const GemmSide& s, int64_t w, int64_t count)
{
    if (!s.partials)
        return;
    const int lane = threadIdx.x % 32;
    for (int64_t column = 32 * w + lane; column < s.columns; column += 32 * count) {
        float sum = 0.0f;
#pragma unroll 16
        for (int32_t i = 0; i < s.strips; ++i)
            sum += __ldcg(s.partials + i * s.columns + column);
        store_as(s.out, column, s.dtype, s.add ? sum + load_as(s.out, column, s.dtype) : sum);
    }
}

// E, E2: the products' epilogues (E2 void: one product).  E::Params is its
// arguments.  An object of E is made for each tile and thread by E(params,
// shape, row, first column, columns, item, which half of the tile's columns, 32 x
// 33 floats of shared memory of the warp's own); it gets the sums of its row by
// chunk(params, shape, column, number of the chunk, values, those floats) and
// ends with end(params, shape).  E::kUnroll chunks are unrolled.
template <typename E>
struct ParamsOf {
    using type = typename E::Params;
};
template <>
struct ParamsOf<void> {
    struct type {};
};
template <int BN, typename E, typename E2>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    k_gemm(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
           const __grid_constant__ GemmShape shape, const __grid_constant__ typename E::Params e,
           const __grid_constant__ CUtensorMap map_a2, const __grid_constant__ CUtensorMap map_b2,
           const __grid_constant__ GemmShape shape2,
           const __grid_constant__ typename ParamsOf<E2>::type e2, const GemmDeal deal,
           const GemmSide side)
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

    constexpr bool kTwo = !std::is_void_v<E2>;
    // items of the first product
    const int32_t count = deal.longs, pair = int32_t(blockIdx.x / 2);
    int32_t turn = 0, item = gemm_dealt(deal, pair, 0);
    const auto next = [&] { item = gemm_dealt(deal, pair, ++turn); };
    bool ok = true;

    if (warp == 0 && elect_one()) {
        uint32_t stage = 0, phase = 0;
        const uint32_t full_first = in_block(full, 0);
        while (item >= 0) {
            const bool second = kTwo && item >= count;
            const GemmShape& s = second ? shape2 : shape;
            const CUtensorMap* const a = second ? &map_a2 : &map_a;
            const CUtensorMap* const b = second ? &map_b2 : &map_b;
            // of both blocks' tiles
            const uint32_t bytes =
                2 * (R::kBytesA + (s.b_across ? R::kBytesB : R::kRowsB * kGemmInner * 2));
            for (int32_t chain = 0; chain < s.chains && ok; ++chain) {
                const GemmItem it = gemm_item(s, second ? item - count : item, chain);
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
                        load_tile(to, a, inner, row_a, bar);
                    } else {
                        load_tile(to, a, row_a, inner, bar);
                        load_tile(to + 8192, a, row_a + 64, inner, bar);
                    }
                    if (!s.b_across) {
                        load_tile(to + R::kBytesA, b, inner, row_b, bar);
                    } else {
#pragma unroll
                        for (int i = 0; i < R::kRowsB; i += 64)
                            load_tile(to + R::kBytesA + i * 128, b, row_b + i, inner, bar);
                    }
                    if (++stage == R::kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok)
                break;
            next();
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
        int32_t n = 0;
        while (item >= 0) {
            const bool second = kTwo && item >= count;
            const GemmShape& s = second ? shape2 : shape;
            const uint32_t step_a = s.a_across ? 2048 : 32, step_b = s.b_across ? 2048 : 32;
            for (int32_t chain = 0; chain < s.chains && ok; ++chain, ++n) {
                const GemmItem it = gemm_item(s, second ? item - count : item, chain);
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
            if (!ok)
                break;
            next();
        }
    } else if (warp == 3) {
        gemm_side(side, blockIdx.x, gridDim.x);
    } else if (warp >= 4) {
        constexpr int kHalf = BN / 2, kChunk = kHalf < 32 ? kHalf : 32;
        const uint32_t quarter = warp % 4, half = (warp - 4) / 4;
        const uint32_t done = in_block(sums_empty, 0);
        float* const stage = reinterpret_cast<float*>(
            raw + (ring - smem_address(raw)) + R::kStages * R::kStage + (warp - 4) * R::kWarpStage);
        int32_t n = 0;
        // One tile by the epilogue F; false if a wait ran out.
        const auto tile = [&](auto* kind, const GemmShape& s, const auto& params, int32_t which,
                              int32_t chain) {
            using F = std::remove_pointer_t<decltype(kind)>;
            const GemmItem it = gemm_item(s, which, chain);
            const int32_t slot = n & 1;
            const int32_t row = it.m0 + 128 * int32_t(rank) + 32 * int32_t(quarter) +
                                int32_t(threadIdx.x % 32);
            const int32_t column = it.tile_n * BN + kHalf * int32_t(half);
            F epilogue(params, s, row, column, kHalf, it, int32_t(half), stage);
            const bool there = barrier_wait(sums_full + 8 * slot, (n >> 1) & 1, dead);
            if (!__all_sync(0xFFFFFFFFu, there))
                return false;
            after_sync();
            const uint32_t from = tmem + uint32_t(slot * R::kAccColumns) + half * kHalf +
                                  ((32 * quarter) << 16);
            constexpr int kUnroll = F::kUnroll;
#pragma unroll kUnroll
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
                epilogue.chunk(params, s, column + c * kChunk, c, v, stage);
            }
            epilogue.end(params, s);
            __syncwarp();
            ++n;
            return true;
        };
        while (item >= 0) {
            if (!kTwo || item < count) {
                for (int32_t chain = 0; chain < shape.chains && ok; ++chain)
                    ok = tile(static_cast<E*>(nullptr), shape, e, item, chain);
            }
            if constexpr (kTwo)
                if (item >= count)
                    for (int32_t chain = 0; chain < shape2.chains && ok; ++chain)
                        ok = tile(static_cast<E2*>(nullptr), shape2, e2, item - count, chain);
            if (!ok)
                break;
            next();
        }
    }
    __syncwarp();
    before_sync();
    __syncthreads();
    cluster_sync();
    after_sync();
    if (warp == 2)
        tmem_free(tmem, R::kColumns);
    if (threadIdx.x == 0 && *dead && shape.gave_up)
        *static_cast<volatile int32_t*>(shape.gave_up) = 1;
}

// One product as the kernel takes it.
template <typename E>
struct GemmPart {
    CUtensorMap a, b;
    GemmShape s{};  // all zero: none
    typename ParamsOf<E>::type e{};
};
// Fills in what follows from the operands; s has the splits and chains.
template <int BN, typename E>
inline int gemm_part(const GemmOperand& a, const GemmOperand& b, GemmShape s, bool bf16,
                     const typename E::Params& e, GemmPart<E>* part)
{
    int rc = gemm_map(a, 128, bf16, &part->a);
    if (rc == cudaSuccess)
        rc = gemm_map(b, BN / 2, bf16, &part->b);
    s.m = int32_t(a.outer);
    s.n = int32_t(b.outer);
    s.tiles_m = (s.m + kGemmTileM - 1) / kGemmTileM;
    s.tiles_n = (s.n + BN - 1) / BN;
    s.blocks = int32_t((a.inner + kGemmInner - 1) / kGemmInner);
    s.what = mma_what(bf16, a.across, b.across, kGemmTileM, BN);
    s.a_across = a.across;
    s.b_across = b.across;
    part->s = s;
    part->e = e;
    return rc;
}

inline int64_t gemm_items(const GemmShape& s)
{
    return int64_t(s.tiles_m) * s.tiles_n * s.splits;
}
// Launches the items of one or two products; deal: as gemm_deal makes it.
template <int BN, typename E, typename E2>
inline int gemm_launch(const GemmPart<E>& p, const GemmPart<E2>& q, const GemmDeal& deal,
                       const GemmSide& side, cudaStream_t stream)
{
    using R = GemmRing<BN>;
    const cudaError_t err = cudaFuncSetAttribute(
        k_gemm<BN, E, E2>, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kSmem);
    if (err != cudaSuccess)
        return int(err);
    return launch_early(k_gemm<BN, E, E2>, dim3(unsigned(2 * deal.pairs)), kGemmThreads, R::kSmem,
                        stream, p.a, p.b, p.s, p.e, q.a, q.b, q.s, q.e, deal, side);
}
template <int BN, typename E>
inline int gemm_run(const GemmOperand& a, const GemmOperand& b, const GemmShape& s, bool bf16,
                    const typename E::Params& e, const GemmSide& side, int sm_count,
                    cudaStream_t stream)
{
    GemmPart<E> p;
    const int rc = gemm_part<BN, E>(a, b, s, bf16, e, &p);
    if (rc != cudaSuccess)
        return rc;
    GemmPart<void> none;
    none.a = p.a;
    none.b = p.b;
    const int64_t items = gemm_items(p.s);
    if (items >= int64_t(1) << 30)
        return int(cudaErrorInvalidValue);
    const int pairs = int(items < sm_count / 2 ? items : sm_count / 2);
    return gemm_launch<BN, E, void>(p, none, GemmDeal{pairs, int32_t(items), 0, 0, 0, 0}, side,
                                    stream);
}

}  // namespace detail
}  // namespace osr
