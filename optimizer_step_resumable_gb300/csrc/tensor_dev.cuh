// tensor_dev.cuh -- the instructions that move tiles into shared memory and
// through the tensor cores of sm_103a: mbarriers, tiled bulk copies, tcgen05.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace osr {
namespace detail {

__device__ __forceinline__ uint32_t smem_address(const void* p)
{
    return uint32_t(__cvta_generic_to_shared(p));
}
// The same place in the shared memory of block `rank` of the cluster.
__device__ __forceinline__ uint32_t in_block(uint32_t address, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(address), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
__device__ __forceinline__ bool elect_one()
{
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(is));
    return is != 0;
}

// ---- mbarriers ------------------------------------------------------------
__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void barriers_visible()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
// `bar`: an address in the cluster's shared memory (in_block).  What the barriers
// here guard between the blocks of a pair is tensor memory, whose operations have
// fences of their own (before_sync, after_sync), and no writes to memory: so the
// arrival is relaxed and does not wait for the warp's stores (8192 rows, 768 to
// 768: 16.7 us against 18.0; a backward of 1001 x 509 and 10007 words: 65 against
// 70, the inputs read from memory; no difference where the products are long).
__device__ __forceinline__ void barrier_arrive_at(uint32_t bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}
__device__ __forceinline__ bool barrier_try(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}
__device__ __forceinline__ uint64_t nanoseconds()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// No wait is endless: one that lasts four seconds (the longest that a kernel
// here can need is some milliseconds) gives up, says so in *dead, at which
// every other wait of the block ends too, and returns false.
constexpr uint64_t kPatience = 4000000000ull;

static __device__ __noinline__ bool barrier_wait_long(uint32_t bar, uint32_t parity,
                                                      volatile int* dead)
{
    const uint64_t begin = nanoseconds();
    while (!barrier_try(bar, parity)) {
        if (*dead)
            return false;
        if (nanoseconds() - begin > kPatience) {
            *dead = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool barrier_wait(uint32_t bar, uint32_t parity, volatile int* dead)
{
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
        if (barrier_try(bar, parity))
            return true;
    return barrier_wait_long(bar, parity, dead);
}

// ---- tiled copies ---------------------------------------------------------
// A tile of a matrix into this block's shared memory, counted by the barrier
// `bar` of either block of a pair.
__device__ __forceinline__ void load_tile(uint32_t to, const CUtensorMap* map, int x, int y,
                                          uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 ".cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(to),
                 "l"(map), "r"(bar), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- tcgen05 --------------------------------------------------------------
// Tensor memory is allocated and freed by one warp of each block of the pair.
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t address, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(address),
                 "r"(columns));
}
__device__ __forceinline__ void before_sync()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void after_sync()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// d (+)= a b for a tile of both blocks; 16 of the inner dimension.
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t what,
                                         bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(what), "r"(uint32_t(add))
                 : "memory");
}
// Arrives at `bar` of both blocks when all products issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                 ".multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"(uint16_t(3))
                 : "memory");
}
// Thread l of a warp gets C columns of lane 32 (warp mod 4) + l.  The values
// are there after tmem_wait, which every use of them has to follow: so it
// takes them as operands.
template <int C>
__device__ __forceinline__ void tmem_read(uint32_t address, float (&v)[C])
{
    static_assert(C == 16 || C == 32, "");
    if constexpr (C == 32)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
            "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
            : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
              "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
              "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
              "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
              "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]),
              "=f"(v[30]), "=f"(v[31])
            : "r"(address));
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
              "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
              "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
            : "r"(address));
}
template <int C>
__device__ __forceinline__ void tmem_wait(float (&v)[C])
{
    if constexpr (C == 32)
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                       "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                       "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]),
                       "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]),
                       "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]),
                       "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
                     :
                     : "memory");
    else
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                       "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                       "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                     :
                     : "memory");
}

// What a tile in shared memory looks like to the tensor cores: rows of 128
// bytes, 16-byte pieces swizzled within eight rows, as the tiled copies leave
// them.  A tile whose inner dimension lies along the rows has its eight-row
// groups 1024 bytes apart; one whose inner dimension goes from row to row has
// those too, and 64 outer elements a row, the next 64 `outer` bytes further
// on.
__device__ __forceinline__ uint64_t tile_descriptor(uint32_t address, uint32_t outer)
{
    return uint64_t((address & 0x3FFFF) >> 4) | (uint64_t(outer >> 4) << 16) |
           (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// kind::f16 with float32 sums; m, n: the pair's tile; *_across: the inner
// dimension goes from row to row.
__host__ __device__ inline uint32_t mma_what(bool bf16, bool a_across, bool b_across, int m, int n)
{
    const uint32_t t = bf16 ? 1 : 0;
    return (1u << 4) | (t << 7) | (t << 10) | (uint32_t(a_across) << 15) |
           (uint32_t(b_across) << 16) | (uint32_t(n / 8) << 17) | (uint32_t(m / 16) << 24);
}

}  // namespace detail
}  // namespace osr
