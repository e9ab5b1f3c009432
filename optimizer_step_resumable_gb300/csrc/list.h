// list.h -- the step over a list of tensors: what its entry points
// (list_api.cu) and its kernels (list_step.cu) share.  Not part of the ABI.
#pragma once

#include <cstdint>

#include "internal.h"

namespace osr {

// 8-bit states keep one scale per block of this many elements of a tensor.
constexpr int kBlockElems = ADAMW_STATE_BLOCK;

// A block's unit of work: up to 8 consecutive blocks of elements of one
// tensor, one for each of its warps.
constexpr int kUnitBlocks = 8;
constexpr int kUnitElems = kUnitBlocks * kBlockElems;

constexpr uint32_t kListDecay = 1u;  // weight decay applies
constexpr uint32_t kListVec = 2u;    // every array at its vector alignment

// One tensor of the list, in device memory.
struct alignas(16) ListTensor {
    float* w;
    void* g;
    void* m;
    void* v;
    float* m_scale;  // 8-bit states: one per block
    float* v_scale;
    void* w_lp;      // 16-bit copy of the weights, or NULL
    int64_t block0;  // blocks of the tensors before it: its place in the random sequence
    int32_t numel;
    uint32_t flags;
    uint64_t pad;  // a multiple of 16 bytes
};

// Unit u covers elements [unit * kUnitElems, ...) of tensor `tensor`.  The
// units of tensors with 32-bit states come first, in the tensors' order.
struct ListUnit {
    int32_t tensor;
    int32_t unit;
};

struct ListView {
    const ListTensor* tensors;
    const ListUnit* units;
    int32_t n_units;
};

// Blocks of the norm reduction: a function of the number of units alone, so
// that the order of the sum, and with it every bit of the norm, is too.
inline int list_norm_blocks(int32_t n_units)
{
    return n_units < 1 ? 1 : n_units > kNormBlocksMax ? kNormBlocksMax : n_units;
}

// Per-block partial sums of g^2 over the list (8 bytes per block).
int launch_list_norm(const ListView& list, int32_t g_dtype, double* partials, void* stream);
// Blocks that the current device keeps resident, of the update of each kind
// of state.
struct ListBlocks {
    int32_t plain, eight;
};
int list_step_blocks(int32_t g_dtype, int sm_count, ListBlocks* most);
// The update of the units with 32-bit (plain) and with 8-bit states; k.fin
// finishes the norm from the partials.  key: the random numbers' key of this
// step (8-bit states).
int launch_list_step(const ListView& plain, const ListView& eight, int32_t g_dtype,
                     int32_t w_lp_dtype, const StepScalars& k, uint32_t key, bool zero_grad,
                     const ListBlocks& most, void* stream);

// The 32-bit hash behind the random rounding: xor-shifts and odd multipliers
// (the first two of the 32-bit primes published with xxHash), each invertible,
// so distinct words stay distinct.
#ifdef __CUDACC__
#define OSR_BOTH __host__ __device__
#else
#define OSR_BOTH
#endif
OSR_BOTH inline uint32_t hash32_begin(uint32_t x) { return x ^ (x >> 16); }
OSR_BOTH inline uint32_t hash32_middle(uint32_t x)
{
    x *= 0x9E3779B1u;
    return (x ^ (x >> 15)) * 0x85EBCA77u;
}
OSR_BOTH inline uint32_t hash32_end(uint32_t x)
{
    x = hash32_middle(x);
    return x ^ (x >> 16);
}
OSR_BOTH inline uint32_t hash32(uint32_t x) { return hash32_end(hash32_begin(x)); }

// The key of step t: the random number of position p is hash32(p ^ key).
inline uint32_t rounding_key(uint32_t seed, int32_t t)
{
    return hash32(hash32(uint32_t(t)) ^ seed);
}

}  // namespace osr
