// list_step.cu -- the clip + AdamW step over a list of tensors, for sm_103a:
// one reduction and one update launch for all tensors of a kind of state,
// whatever their number.
//
// "Training as a Recoverable State Transition" (aihero.club), section "The
// Exact Targets of Clipping and AdamW": the norm of all gradients joined into
// one vector, the clip factor, the AdamW update.  Here the vector is never
// joined: a table of units (up to 2048 consecutive elements of one tensor)
// built once per list tells every block what to work on.
//
// HBM-bound: streams read once and written once.  Bytes per parameter of the
// update with a 16-bit gradient and weight copy: 28 with 32-bit states (w 8,
// m and v 16, g 2, copy 2), 16.06 with 8-bit ones (w 8, m and v 4, scales
// 16/256, g 2, copy 2); the norm reads g once more.  On GB300, 110M
// parameters in 196 tensors: 491 us and 325 us a step (the copy's bandwidth
// would take 489 and 294 for these bytes); 570M in 8 bits 1620 us (1523).  The
// norm kernel's share is 46 us: 33 for g, the rest for writing back what the
// step before left in L2.
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "adamw_dev.cuh"
#include "common.cuh"
#include "early_dev.cuh"
#include "list.h"
#include "norm_dev.cuh"
#include "state8_dev.cuh"

namespace osr {
namespace {

constexpr int kStepThreads = kUnitElems / (kBlockElems / 32);
constexpr int kLane = kBlockElems / 32;  // elements of a block per lane

// A lane's kLane elements of a block are adjacent: lane * kLane, ...  In a
// vector access a lane moves all of them (32 bytes of float32 in one
// instruction), and a warp's accesses lie in a row.  (Two 16-byte accesses
// half a block apart: 389 us instead of 351 for 110M parameters in 8 bits.)

// ---------------------------------------------------------------------------
// The norm.
// ---------------------------------------------------------------------------

// A sum of two floats, hi the rounded one: 48 bits.  Binary64 additions run at
// 1/64 of float32's rate: with them a third of the norm kernel's time went into
// a thread's sums, and joining the threads' and the blocks' sums took 1 to 2 us
// of every step (a million elements in 8 bits: 14.5 us, not 12.4).
struct Sum2 {
    float hi, lo;
};
__device__ __forceinline__ Sum2 add(Sum2 a, Sum2 b)
{
    const float s = __fadd_rn(a.hi, b.hi);
    const float back = __fsub_rn(s, a.hi);
    // s + e is the exact sum of the his
    const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, back)), __fsub_rn(b.hi, back));
    const float lo = __fadd_rn(e, __fadd_rn(a.lo, b.lo));
    const float hi = __fadd_rn(s, lo);
    return Sum2{hi, __fsub_rn(lo, __fsub_rn(hi, s))};
}

// A partial sum of squares, in 8 bytes: a Sum2 or, with the top bit set, a
// binary64 number, for what float32 does not hold.
__device__ __forceinline__ uint2 pack(Sum2 s)
{
    return make_uint2(__float_as_uint(s.lo), __float_as_uint(s.hi));
}
__device__ __forceinline__ uint2 pack(double d)
{
    return make_uint2(uint32_t(__double2loint(d)), uint32_t(__double2hiint(d)) | 0x80000000u);
}
__device__ __forceinline__ bool is_double(uint2 p) { return p.y >> 31; }
__device__ __forceinline__ Sum2 sum_of(uint2 p)
{
    return Sum2{__uint_as_float(p.y), __uint_as_float(p.x)};
}
__device__ __forceinline__ double value_of(uint2 p)
{
    return is_double(p) ? __hiloint2double(int(p.y & 0x7fffffffu), int(p.x))
                        : double(__uint_as_float(p.y)) + double(__uint_as_float(p.x));
}
// The sum over the first kLanes lanes of a warp, in lane 0.  more, and its
// binary64 share, where any lane has one.
template <int kLanes>
__device__ __forceinline__ uint2 warp_sum(Sum2 s, bool more, double share)
{
    if (__any_sync(0xffffffffu, more)) {
        share += double(s.hi) + double(s.lo);
#pragma unroll
        for (int d = kLanes / 2; d > 0; d >>= 1)
            share += __shfl_down_sync(0xffffffffu, share, d);
        return pack(share);
    }
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1)
        s = add(s, Sum2{__shfl_down_sync(0xffffffffu, s.hi, d),
                        __shfl_down_sync(0xffffffffu, s.lo, d)});
    return pack(s);
}
// The sum over a block, in thread 0; called once in a kernel.
template <int kThreads>
__device__ __forceinline__ uint2 block_sum(Sum2 s, bool more, double share)
{
    constexpr int kWarps = kThreads / 32;
    __shared__ uint2 warps[kWarps];
    const int lane = threadIdx.x & 31;
    uint2 p = warp_sum<32>(s, more, share);
    if (lane == 0)
        warps[threadIdx.x >> 5] = p;
    __syncthreads();
    if (threadIdx.x < 32) {
        p = lane < kWarps ? warps[lane] : make_uint2(0u, 0u);
        more = is_double(p);
        p = warp_sum<kWarps>(more ? Sum2{0.0f, 0.0f} : sum_of(p), more, more ? value_of(p) : 0.0);
    }
    return p;
}

// Level 1 of the norm.  Block b takes the contiguous units [U b / P,
// U (b + 1) / P), tensor by tensor: within a tensor it streams, with no table
// between two loads.  Each thread has two sets of kSet loads, one on the way
// while the other is summed: a run of normdev::run_sumsq.  Default L2
// priority: the update reads g next.
template <typename G>
__global__ void __launch_bounds__(kNormThreads, 4)
    k_list_norm(ListView list, uint2* __restrict__ partials)
{
    constexpr int kSet = sizeof(G) == 2 ? 4 : 2;
    constexpr int kTile = kNormThreads * kLane;  // elements of the block's one load
    const int32_t lo = int32_t(int64_t(list.n_units) * blockIdx.x / gridDim.x);
    const int32_t hi = int32_t(int64_t(list.n_units) * (blockIdx.x + 1) / gridDim.x);
    Sum2 acc{0.0f, 0.0f};
    bool more = false;  // runs that float32 does not hold
    double share = 0.0;
    for (int32_t u = lo; u < hi;) {
        const ListUnit unit = list.units[u];
        const ListTensor& t = list.tensors[unit.tensor];
        const int32_t e0 = unit.unit * kUnitElems, left = t.numel - e0;
        const int32_t units = (left - 1) / kUnitElems + 1;  // to the tensor's end
        const int32_t mine = units < hi - u ? units : hi - u;
        const int32_t end = mine < units ? mine * kUnitElems : left;
        if (u == lo) {  // the tables are no kernel's output
            detail::wait_before();
            detail::go_ahead();
        }
        u += mine;
        const G* const g = static_cast<const G*>(t.g) + e0;
        const bool aligned = t.flags & kListVec;
        int32_t i = int32_t(threadIdx.x) * kLane;
        detail::Raw8<G> x[2][kSet];
        constexpr int32_t kSpan = kSet * kTile;
        auto load = [&](detail::Raw8<G>(&to)[kSet]) {
#pragma unroll
            for (int p = 0; p < kSet; ++p, i += kTile)
                if (aligned && end - i >= kLane)
                    to[p] = detail::load8_cg(g + i);
                else if (end > i)
                    to[p] = detail::load8_part(g + i, end - i);
                else
                    to[p] = detail::Raw8<G>{};
        };
        auto sum = [&](const detail::Raw8<G>(&from)[kSet], int32_t begin) {
            if (begin + int32_t(threadIdx.x) * kLane >= end)
                return;  // nothing of it is this thread's
            float4 y[2 * kSet];
#pragma unroll
            for (int p = 0; p < kSet; ++p)
                detail::widen8(from[p], y[2 * p], y[2 * p + 1]);
            float r;
            if (normdev::run_sumsq_fast<2 * kSet>(y, r) && r <= 0x1p80f) {  // below 2^128 in all
                const float next = __fadd_rn(acc.hi, r);
                const float back = __fsub_rn(next, acc.hi);
                acc.lo = __fadd_rn(acc.lo, __fadd_rn(__fsub_rn(acc.hi, __fsub_rn(next, back)),
                                                     __fsub_rn(r, back)));
                acc.hi = next;
            } else {
                const double d = normdev::run_sumsq<2 * kSet>(y);
                if (__double2hiint(d) | __double2loint(d)) {  // not a run of zeros
                    share += d;
                    more = true;
                }
            }
        };
        load(x[0]);
        for (int32_t done = 0; done < end; done += 2 * kSpan) {
            if (done + kSpan < end)
                load(x[1]);
            sum(x[0], done);
            if (done + 2 * kSpan < end)
                load(x[0]);
            if (done + kSpan < end)
                sum(x[1], done + kSpan);
        }
    }
    if (lo == hi)
        detail::wait_before();
    const uint2 p = block_sum<kNormThreads>(acc, more, share);
    if (threadIdx.x == 0)
        partials[blockIdx.x] = p;
}

// ---------------------------------------------------------------------------
// The update.
// ---------------------------------------------------------------------------

// A thread's share of a block: what it reads.
template <bool k8>
struct Moments;
template <>
struct Moments<false> {
    float m[kLane], v[kLane];
};
template <>
struct Moments<true> {
    uint32_t m[kLane / 4], v[kLane / 4];  // four values a word
    float m_scale, v_scale;
};

// i: the lane's first element; left: from there to the end of the tensor.
template <typename G, bool k8>
__device__ __forceinline__ void load_block(const ListTensor& t, int32_t i, int32_t left, bool vec,
                                           float (&w)[kLane], float (&g)[kLane], Moments<k8>& s)
{
    const float* const wp = t.w + i;
    const G* const gp = static_cast<const G*>(t.g) + i;
    using State = typename std::conditional<k8, uint8_t, float>::type;
    const State* const mp = static_cast<const State*>(t.m) + i;
    const State* const vp = static_cast<const State*>(t.v) + i;
    if (vec) {
        const detail::Raw8<float> a = detail::load8_cs(wp);
        const detail::Raw8<G> b = detail::load8_cs(gp);
        if constexpr (k8) {
            const uint2 c = __ldcs(reinterpret_cast<const uint2*>(mp));
            const uint2 d = __ldcs(reinterpret_cast<const uint2*>(vp));
            s.m[0] = c.x, s.m[1] = c.y, s.v[0] = d.x, s.v[1] = d.y;
        } else {
            const detail::Raw8<float> c = detail::load8_cs(mp), d = detail::load8_cs(vp);
            detail::widen8(c, s.m);
            detail::widen8(d, s.v);
        }
        detail::widen8(a, w);
        detail::widen8(b, g);
    } else {
        if constexpr (k8)
            s.m[0] = s.m[1] = s.v[0] = s.v[1] = 0u;
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            const bool in = j < left;
            w[j] = in ? wp[j] : 0.0f;
            g[j] = in ? detail::load1(gp + j) : 0.0f;
            if constexpr (k8) {
                s.m[j >> 2] |= in ? uint32_t(mp[j]) << (8 * (j & 3)) : 0u;
                s.v[j >> 2] |= in ? uint32_t(vp[j]) << (8 * (j & 3)) : 0u;
            } else {
                s.m[j] = in ? mp[j] : 0.0f;
                s.v[j] = in ? vp[j] : 0.0f;
            }
        }
    }
    if constexpr (k8) {
        s.m_scale = left > 0 ? t.m_scale[i / kBlockElems] : 0.0f;
        s.v_scale = left > 0 ? t.v_scale[i / kBlockElems] : 0.0f;
    }
}

// When an update cannot be seen in w.  |m| < tiny makes it at most `most`
// whatever v is: with u = round(step_size round(m / denom)), denom >= eps,
// every step monotone, most = round(step_size round(2^-100 / eps)).  tiny is
// 2^-100, or 0 where that bound is no number (eps = 0).
struct Unseen {
    float tiny, most;
};

// adamw_elem's bits, without its root and quotient for moments that have died
// away (rows no token has touched for hundreds of steps) or never lived: those
// two take a slow path for zeros and subnormal numbers (110M parameters of
// dead m, or of zeros: 598 and 504 us, not 492).  If w d - most and w d + most round to the same
// number, so does w d - u for every u between; for m = 0, u is 0.
__device__ __forceinline__ void adamw_elem_any(float& w, float g, float& m, float& v, float s,
                                               const StepScalars& k, float d, const Unseen& un)
{
    const float gh = __fmul_rn(g, s);
    const float m1 = __fmaf_rn(k.beta1, m, __fmul_rn(k.omb1, gh));
    const float v1 = __fmaf_rn(k.beta2, v, __fmul_rn(__fmul_rn(k.omb2, gh), gh));
    if (fabsf(m1) < un.tiny && v1 >= 0.0f) {
        const float most = m1 == 0.0f ? 0.0f : un.most;
        const float low = __fmaf_rn(w, d, -most), high = __fmaf_rn(w, d, most);
        if (__float_as_uint(low) == __float_as_uint(high)) {
            w = low;
            m = m1;
            v = v1;
            return;
        }
    }
    adamwdev::adamw_elem(w, g, m, v, s, k, d);
}

// The update of a block, in registers.  8-bit states: m, v become the new
// bytes and scales; everything past the end of a partial block is 0 and
// leaves the block's largest values alone.
__device__ __forceinline__ void update_block(const ListTensor&, int32_t, float (&w)[kLane],
                                             const float (&g)[kLane], Moments<false>& x, float s,
                                             const StepScalars& k, float d, uint32_t,
                                             const Unseen& un)
{
#pragma unroll
    for (int j = 0; j < kLane; ++j)
        adamw_elem_any(w[j], g[j], x.m[j], x.v[j], s, k, d, un);
}
__device__ __forceinline__ void update_block(const ListTensor& t, int32_t i, float (&w)[kLane],
                                             const float (&g)[kLane], Moments<true>& x, float s,
                                             const StepScalars& k, float d, uint32_t key,
                                             const Unseen&)
{
    // A scale is a power of two, so beta times the scale times the value is
    // rounded as beta times the widened value is.
    const float b1 = __fmul_rn(k.beta1, x.m_scale), b2 = __fmul_rn(k.beta2, x.v_scale);
    float m[kLane], v[kLane];
    float m_most = 0.0f, v_most = 0.0f;
#pragma unroll
    for (int j = 0; j < kLane; j += 2) {
        state8::moments(packed::mul2(make_float2(g[j], g[j + 1]), packed::both(s)),
                        state8::widen_m((x.m[j >> 2] >> (8 * (j & 3))) & 0xffffu),
                        state8::widen_v((x.v[j >> 2] >> (8 * (j & 3))) & 0xffffu), b1, b2, k,
                        m + j, v + j);
        m_most = state8::largest(m_most, fabsf(m[j]), fabsf(m[j + 1]));
        v_most = state8::largest(v_most, v[j], v[j + 1]);
    }
    // non-negative floats order as their bits do, infinity and NaN above all
    uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(m_most));
    uint32_t vb = __reduce_max_sync(0xffffffffu, __float_as_uint(v_most));
    const bool fast = mb < state8::kMFast && vb < state8::kVFast;  // the same in every lane
    if (mb >= state8::kInfinity || vb >= state8::kInfinity) {
        mb = vb = 0u;
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            const uint32_t a = __float_as_uint(fabsf(m[j])), b = __float_as_uint(v[j]);
            mb = a < state8::kInfinity && a > mb ? a : mb;
            vb = b < state8::kInfinity && b > vb ? b : vb;
        }
        mb = __reduce_max_sync(0xffffffffu, mb);
        vb = __reduce_max_sync(0xffffffffu, vb);
    }
    const uint32_t me = state8::scale_exponent(mb, state8::kMTop);
    const uint32_t ve = state8::scale_exponent(vb, state8::kVTop);
    x.m_scale = state8::scale_of(me);
    x.v_scale = state8::scale_of(ve);
    // The random numbers: the hash of position ^ key.  The elements of a lane
    // differ in the lowest three bits only, which the hash's first step
    // (x ^ x >> 16) leaves in place: it is done once for all of them.
    const uint64_t p0 = uint64_t(t.block0) * kBlockElems + uint32_t(i);
    const uint32_t first = hash32_begin(uint32_t(p0) ^ key ^
                                        (uint32_t(p0 >> 32) * 0x9E3779B1u));
    const float inv = fast ? k.inv_sqrt_bc2 * state8::kRootUnit : k.inv_sqrt_bc2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r[j] = first ^ uint32_t(4 * h + j);
        const float* const mh = m + 4 * h;
        const float* const vh = v + 4 * h;
        float* const wh = w + 4 * h;
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const float2 v2 = make_float2(vh[j], vh[j + 1]);
            const float2 root = fast ? state8::root_fast(v2)
                                     : make_float2(__fsqrt_rn(v2.x), __fsqrt_rn(v2.y));
            const float2 wn = state8::weight(make_float2(wh[j], wh[j + 1]),
                                             make_float2(mh[j], mh[j + 1]), root, inv, k, d);
            wh[j] = wn.x, wh[j + 1] = wn.y;
        }
        if (fast) {
            state8::narrow4(mh, state8::move_m(me), vh, state8::move_v(ve), r, x.m[h], x.v[h]);
        } else {
            x.m[h] = x.v[h] = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t hash = hash32_end(r[j]);
                x.m[h] |= state8::narrow_m(mh[j], state8::inverse_of(me), hash) << (8 * j);
                x.v[h] |= state8::narrow_v(vh[j], state8::inverse_of(ve), hash) << (8 * j);
            }
        }
    }
}

template <typename G, bool k8>
__device__ __forceinline__ void store_block(const ListTensor& t, int32_t i, int32_t left, bool vec,
                                            const float (&w)[kLane], const Moments<k8>& s,
                                            bool zero_grad, int32_t w_lp_dtype)
{
    float* const wp = t.w + i;
    G* const gp = static_cast<G*>(t.g) + i;
    using State = typename std::conditional<k8, uint8_t, float>::type;
    State* const mp = static_cast<State*>(t.m) + i;
    State* const vp = static_cast<State*>(t.v) + i;
    if (vec) {
        detail::store8_cs(wp, w);
        if constexpr (k8) {
            __stcs(reinterpret_cast<uint2*>(mp), make_uint2(s.m[0], s.m[1]));
            __stcs(reinterpret_cast<uint2*>(vp), make_uint2(s.v[0], s.v[1]));
        } else {
            detail::store8_cs(mp, s.m);
            detail::store8_cs(vp, s.v);
        }
        if (t.w_lp && w_lp_dtype == kDtypeF16)
            detail::store8_cs(static_cast<__half*>(t.w_lp) + i, w);
        else if (t.w_lp)
            detail::store8_cs(static_cast<__nv_bfloat16*>(t.w_lp) + i, w);
        if (zero_grad) {
            const float zero[kLane] = {};
            detail::store8_cs(gp, zero);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            if (j >= left)
                continue;
            wp[j] = w[j];
            if constexpr (k8) {
                mp[j] = uint8_t(s.m[j >> 2] >> (8 * (j & 3)));
                vp[j] = uint8_t(s.v[j >> 2] >> (8 * (j & 3)));
            } else {
                mp[j] = s.m[j];
                vp[j] = s.v[j];
            }
            if (t.w_lp && w_lp_dtype == kDtypeF16)
                detail::store1_lp(static_cast<__half*>(t.w_lp) + i + j, w[j]);
            else if (t.w_lp)
                detail::store1_lp(static_cast<__nv_bfloat16*>(t.w_lp) + i + j, w[j]);
            if (zero_grad)
                detail::store1_zero(gp + j);
        }
    }
}

// The update of the list's units of one kind of state.  Every block first
// adds the norm's partials up in the same fixed order (the same bits
// everywhere; block 0 of the kernel that runs first publishes the result),
// as the fused kernel of the flat state does, while its first unit's inputs
// are on their way.  Before the wait only the tables are read, which no kernel
// writes: that the kernels before the norm have completed when this one starts
// does not make what they wrote (w, m, v, g, the counters) visible to it; its
// own wait does.
//
// A block takes one unit after another, a warp of it one block of elements.
// Its first warp keeps the tables ahead of it through shared memory: in the
// round of unit i it asks for the tensor of unit i + 2, the table entry of
// unit i + 3 and the number of unit i + 4, each known from an earlier round,
// so no round waits for a chain of loads, and the pointers take no
// registers.  Long lists hand the units out by a counter, which keeps the
// blocks close to one another in memory.  That closeness is what the update
// lives on: units of 4096 or 8192 elements, or a ring with the next unit's
// inputs on their way (cp.async), which widen the stretch of memory in flight,
// took 423 and 369 us where this form took 334 (110M parameters, 8 bits).
constexpr int kRing = 4;

template <int kBytes>
__device__ __forceinline__ void copy_async(void* to, const void* from)
{
    const uint32_t d = uint32_t(__cvta_generic_to_shared(to));
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(from), "n"(kBytes)
                     : "memory");
}

template <typename G, bool k8>
__global__ void __launch_bounds__(kStepThreads, 4)
    k_list_step(ListView list, StepScalars k, Unseen un, uint32_t key, bool publish,
                bool zero_grad, int32_t w_lp_dtype)
{
    const int lane = threadIdx.x & 31;
    const int32_t lane_e0 = int32_t(threadIdx.x >> 5) * kBlockElems + lane * kLane;
    __shared__ ListTensor s_tensor[kRing];
    __shared__ ListUnit s_unit[kRing];  // unit < 0: no more
    __shared__ float s_scale;
    __shared__ int s_skip;
    __shared__ float s_block_scales[2][2][kUnitBlocks];
    uint32_t* const ctr = k.chunk_ctr;
    const int32_t grid = int32_t(gridDim.x);
    auto ask_unit = [&](int slot, int32_t u) {  // one lane
        if (u < list.n_units)
            copy_async<8>(&s_unit[slot], list.units + u);
        else
            s_unit[slot] = ListUnit{0, -1};
    };
    auto ask_tensor = [&](int slot) {  // a warp
        constexpr int kWords = int(sizeof(ListTensor) / 16);
        const ListUnit unit = s_unit[slot];
        if (unit.unit >= 0 && lane < kWords)
            copy_async<16>(reinterpret_cast<uint4*>(&s_tensor[slot]) + lane,
                           reinterpret_cast<const uint4*>(list.tensors + unit.tensor) + lane);
    };
    // the first units are those of a plain stride; the counter goes on from there
    int32_t u = int32_t(blockIdx.x) + (kRing - 1) * grid;  // number of unit i + 3
    if (threadIdx.x < 32) {
        if (lane < kRing - 1)
            ask_unit(lane, int32_t(blockIdx.x) + lane * grid);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        ask_tensor(0);
        ask_tensor(1);
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    float s = 0.0f;
    int32_t done = -1;  // the unit before
    for (int i = 0;; ++i) {
        __syncthreads();
        if (k8 && done >= 0 && threadIdx.x >= kStepThreads - 32 && lane < 2 * kUnitBlocks) {
            // The block scales of the unit before, all of one moment in one
            // store: one 4-byte store a warp, each a partial write of a
            // sector that the neighbours write too, cost 50 of 280 us.
            const ListTensor& p = s_tensor[(i + kRing - 1) % kRing];
            const int32_t b = done * kUnitBlocks + lane % kUnitBlocks;
            if (b <= (p.numel - 1) / kBlockElems)
                (lane < kUnitBlocks ? p.m_scale : p.v_scale)[b] =
                    s_block_scales[(i + 1) & 1][lane / kUnitBlocks][lane % kUnitBlocks];
        }
        const ListTensor& t = s_tensor[i % kRing];
        const int32_t unit = s_unit[i % kRing].unit;
        const int32_t e = unit * kUnitElems + lane_e0;  // the lane's first element
        const int32_t left = unit < 0 ? 0 : t.numel - e;
        const bool vec = left >= kLane && (t.flags & kListVec);
        // whether the warp has any element: its lanes meet in the block's sums
        const bool any = unit >= 0 && left + lane * kLane > 0;
        float w[kLane], g[kLane];
        Moments<k8> x;
        if (i == 0) {
            detail::wait_before();
            detail::go_ahead();
        }
        if (any)
            load_block<G, k8>(t, e, left, vec, w, g, x);
        if (threadIdx.x < 32 && unit >= 0) {
            ask_tensor((i + 2) % kRing);
            if (lane == 0) {
                ask_unit((i + 3) % kRing, u);
                u = !ctr ? u + grid
                    : u < list.n_units ? kRing * grid + int32_t(atomicAdd(ctr, 1u)) : u;
            }
        }
        if (i == 0) {
            Sum2 sum{0.0f, 0.0f};
            bool more = false;
            double share = 0.0;
            for (int q = threadIdx.x; q < k.fin.nparts; q += kStepThreads) {
                const uint2 p = __ldcg(reinterpret_cast<const uint2*>(k.fin.partials) + q);
                if (is_double(p)) {
                    share += value_of(p);
                    more = true;
                } else {
                    sum = add(sum, sum_of(p));
                }
            }
            const uint2 all = block_sum<kStepThreads>(sum, more, share);
            if (threadIdx.x == 0) {
                const double total = value_of(all);
                const bool mine = publish && blockIdx.x == 0;
                const NormResult r = normdev::make_result(total, k.fin.clip, k.fin.grad_scale,
                                                          mine ? k.fin.d_res->seq + 1u : 0u);
                s_scale = r.scale;
                s_skip = r.nonfinite;
                if (mine)
                    normdev::publish(r, k.fin.d_res, k.fin.h_res);
            }
            __syncthreads();
            s = s_scale;
            if (s_skip)
                break;
        }
        if (unit < 0)
            break;
        if (any) {
            update_block(t, e, w, g, x, s, k, (t.flags & kListDecay) ? k.decay : 1.0f, key,
                         un);
            store_block<G, k8>(t, e, left, vec, w, x, zero_grad, w_lp_dtype);
            if constexpr (k8) {
                if (lane == 0) {
                    s_block_scales[i & 1][0][threadIdx.x >> 5] = x.m_scale;
                    s_block_scales[i & 1][1][threadIdx.x >> 5] = x.v_scale;
                }
            }
        }
        done = unit;
        if (threadIdx.x < 32)
            asm volatile("cp.async.wait_all;" ::: "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (ctr && threadIdx.x == 0) {
        // the last block out resets the counters for the next launch
        __threadfence();
        if (atomicAdd(ctr + 1, 1u) == gridDim.x - 1) {
            atomicExch(ctr, 0u);
            atomicExch(ctr + 1, 0u);
        }
    }
}

template <typename G>
int blocks_typed(int sm_count, ListBlocks* most)
{
    cudaError_t e = cudaSuccess;
    most->plain = detail::resident_blocks(reinterpret_cast<const void*>(&k_list_step<G, false>),
                                          kStepThreads, sm_count, &e);
    most->eight = detail::resident_blocks(reinterpret_cast<const void*>(&k_list_step<G, true>),
                                          kStepThreads, sm_count, &e);
    if (e != cudaSuccess)
        cudaGetLastError();  // returned here, not by a later call
    return int(e);
}

template <typename G, bool k8>
int launch_step_typed(const ListView& list, int32_t w_lp_dtype, const StepScalars& k,
                      uint32_t key, bool publish, bool zero_grad, int32_t most, cudaStream_t s)
{
    auto* const kernel = &k_list_step<G, k8>;
    StepScalars kk = k;
    if (int64_t(list.n_units) * kUnitElems < kDynamicChunksMinN)
        kk.chunk_ctr = nullptr;
    const int32_t blocks = list.n_units < 1 ? 1 : list.n_units > most ? most : list.n_units;
    const float bound = k.step_size * (0x1p-100f / k.eps);
    const Unseen un{bound <= FLT_MAX ? 0x1p-100f : 0.0f, bound};
    return detail::launch_early(kernel, dim3(unsigned(blocks)), kStepThreads, 0, s, list, kk, un,
                                key, publish, zero_grad, w_lp_dtype);
}

template <typename G>
int launch_step(const ListView& plain, const ListView& eight, int32_t w_lp_dtype,
                const StepScalars& k, uint32_t key, bool zero_grad, const ListBlocks& most,
                cudaStream_t s)
{
    // a list without elements still publishes its norm; each kernel has its
    // own counters
    StepScalars k8 = k;
    k8.chunk_ctr = k.chunk_ctr + 2;
    // state8::weight takes a subnormal denominator for 0, and 0 / 0 would be NaN
    if (k8.eps > 0.0f && k8.eps < FLT_MIN)
        k8.eps = FLT_MIN;
    int e = cudaSuccess;
    if (plain.n_units > 0 || eight.n_units == 0)
        e = launch_step_typed<G, false>(plain, w_lp_dtype, k, key, true, zero_grad,
                                        most.plain, s);
    if (e == cudaSuccess && eight.n_units > 0)
        e = launch_step_typed<G, true>(eight, w_lp_dtype, k8, key, plain.n_units == 0, zero_grad,
                                       most.eight, s);
    return e;
}

}  // namespace

int launch_list_norm(const ListView& list, int32_t g_dtype, double* partials, void* stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int blocks = list_norm_blocks(list.n_units);
    auto launch = [&](void (*kernel)(ListView, uint2*)) {
        return detail::launch_early(kernel, dim3(unsigned(blocks)), kNormThreads, 0, s, list,
                                    reinterpret_cast<uint2*>(partials));
    };
    if (g_dtype == kDtypeBF16)
        return launch(&k_list_norm<__nv_bfloat16>);
    if (g_dtype == kDtypeF16)
        return launch(&k_list_norm<__half>);
    return launch(&k_list_norm<float>);
}

int list_step_blocks(int32_t g_dtype, int sm_count, ListBlocks* most)
{
    if (g_dtype == kDtypeBF16)
        return blocks_typed<__nv_bfloat16>(sm_count, most);
    if (g_dtype == kDtypeF16)
        return blocks_typed<__half>(sm_count, most);
    return blocks_typed<float>(sm_count, most);
}

int launch_list_step(const ListView& plain, const ListView& eight, int32_t g_dtype,
                     int32_t w_lp_dtype, const StepScalars& k, uint32_t key, bool zero_grad,
                     const ListBlocks& most, void* stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (g_dtype == kDtypeBF16)
        return launch_step<__nv_bfloat16>(plain, eight, w_lp_dtype, k, key, zero_grad, most, s);
    if (g_dtype == kDtypeF16)
        return launch_step<__half>(plain, eight, w_lp_dtype, k, key, zero_grad, most, s);
    return launch_step<float>(plain, eight, w_lp_dtype, k, key, zero_grad, most, s);
}

}  // namespace osr
