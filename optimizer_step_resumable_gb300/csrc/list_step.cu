// list_step.cu -- the clip + AdamW step over a list of tensors, for sm_103a:
// one reduction and one update launch for all of them, whatever their number.
//
// "Training as a Recoverable State Transition" (aihero.club), section "The
// Exact Targets of Clipping and AdamW": the norm of all gradients joined into
// one vector, the clip factor, the AdamW update.  Here the vector is never
// joined: a table of units (up to 1024 consecutive elements of one tensor)
// built once per list gives every warp its work, so a list costs two launches
// and a tensor of one element one warp's unit.
//
// HBM-bound.  Bytes per parameter with a 32-bit gradient: 28 for 32-bit
// states; 16 + 16/256 for 8-bit ones (w 8, g 4, m and v 2 + 2, scales); the
// norm reads g once more, from L2 where it still lies there.
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "adamw_dev.cuh"
#include "common.cuh"
#include "list.h"
#include "norm_dev.cuh"
#include "state8_dev.cuh"

#ifndef MINB
#define MINB 4
#endif
#ifndef NORMB
#define NORMB 4
#endif
#ifndef NRUN
#define NRUN 4
#endif
namespace osr {
namespace {

constexpr int kWarps = kNormThreads / 32;
constexpr int kLane = kBlockElems / 32;  // elements of a block per lane

// Element j (of kLane) of a lane within its block: four consecutive ones and
// four more half a block on (16-byte accesses, a warp's 512 in a row), or, for
// arrays at other alignments and the last block of a tensor, one per stride
// of 32.
__device__ __forceinline__ int element(bool vec, int lane, int j)
{
    return vec ? (j >> 2) * (kBlockElems / 2) + lane * 4 + (j & 3) : j * 32 + lane;
}

__device__ __forceinline__ float4 as_float4(const float (&x)[kLane], int h)
{
    return make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
}
__device__ __forceinline__ void put4(float (&x)[kLane], int h, float4 a)
{
    x[4 * h] = a.x;
    x[4 * h + 1] = a.y;
    x[4 * h + 2] = a.z;
    x[4 * h + 3] = a.w;
}

// ---------------------------------------------------------------------------
// The norm.
// ---------------------------------------------------------------------------

// A lane's gradient elements of one block (`left` elements to the end of the
// tensor; it may be none).
template <typename G>
__device__ __forceinline__ void load_norm(const G* g, bool aligned, int lane, int32_t left,
                                          float4* x)
{
    if (aligned && left >= kBlockElems) {
        x[0] = detail::load4_cg<G>(g + lane * 4);
        x[1] = detail::load4_cg<G>(g + kBlockElems / 2 + lane * 4);
    } else {
        float y[kLane];
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            const int i = j * 32 + lane;
            y[j] = i < left ? detail::load1(g + i) : 0.0f;
        }
        x[0] = make_float4(y[0], y[1], y[2], y[3]);
        x[1] = make_float4(y[4], y[5], y[6], y[7]);
    }
}

// Level 1 of the norm: block b takes units b, b + the grid, ..., kRun at a
// time; a thread's share of them is one run of squares (normdev::run_sumsq),
// added up in double.
constexpr int kRun = NRUN;

template <typename G>
__global__ void __launch_bounds__(kNormThreads, NORMB)
    k_list_norm(ListView list, double* __restrict__ partials)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int32_t warp_e0 = int32_t(threadIdx.x >> 5) * kBlockElems;
    const int32_t stride = int32_t(gridDim.x);
    const ListUnit none{0, -1};
    ListUnit next[kRun];
    int32_t u = int32_t(blockIdx.x);
#pragma unroll
    for (int p = 0; p < kRun; ++p)
        next[p] = u + p * stride < list.n_units ? list.units[u + p * stride] : none;
    double acc = 0.0;
    for (; u < list.n_units; u += kRun * stride) {
        float4 x[2 * kRun];
        ListUnit now[kRun];
#pragma unroll
        for (int p = 0; p < kRun; ++p) {
            now[p] = next[p];
            const int32_t v = u + (p + kRun) * stride;
            next[p] = v < list.n_units ? list.units[v] : none;
        }
#pragma unroll
        for (int p = 0; p < kRun; ++p) {
            const ListTensor& t = list.tensors[now[p].tensor];
            const int32_t e0 = now[p].unit * kUnitElems + warp_e0;
            load_norm<G>(static_cast<const G*>(t.g) + e0, t.flags & kListVec, lane,
                         now[p].unit < 0 ? 0 : t.numel - e0, x + 2 * p);
        }
        acc += normdev::run_sumsq<2 * kRun>(x);
    }
    acc = detail::block_sum<kNormThreads>(acc);
    if (threadIdx.x == 0)
        partials[blockIdx.x] = acc;
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
    uint32_t m[2], v[2];  // four values a word
    float m_scale, v_scale;
};

template <typename G, bool k8>
__device__ __forceinline__ void load_block(const ListTensor& t, int32_t e0, int32_t left, bool vec,
                                           int lane, float (&w)[kLane], float (&g)[kLane],
                                           Moments<k8>& s)
{
    const float* const wp = t.w + e0;
    const G* const gp = static_cast<const G*>(t.g) + e0;
    using State = typename std::conditional<k8, uint8_t, float>::type;
    const State* const mp = static_cast<const State*>(t.m) + e0;
    const State* const vp = static_cast<const State*>(t.v) + e0;
    if (vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = h * (kBlockElems / 2) + lane * 4;
            put4(w, h, __ldcs(reinterpret_cast<const float4*>(wp + i)));
            put4(g, h, detail::load4_cs<G>(gp + i));
            if constexpr (k8) {
                s.m[h] = __ldcs(reinterpret_cast<const uint32_t*>(mp + i));
                s.v[h] = __ldcs(reinterpret_cast<const uint32_t*>(vp + i));
            } else {
                put4(s.m, h, __ldcs(reinterpret_cast<const float4*>(mp + i)));
                put4(s.v, h, __ldcs(reinterpret_cast<const float4*>(vp + i)));
            }
        }
    } else {
        if constexpr (k8)
            s.m[0] = s.m[1] = s.v[0] = s.v[1] = 0u;
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            const int i = j * 32 + lane;
            const bool in = i < left;
            w[j] = in ? wp[i] : 0.0f;
            g[j] = in ? detail::load1(gp + i) : 0.0f;
            if constexpr (k8) {
                s.m[j >> 2] |= in ? uint32_t(mp[i]) << (8 * (j & 3)) : 0u;
                s.v[j >> 2] |= in ? uint32_t(vp[i]) << (8 * (j & 3)) : 0u;
            } else {
                s.m[j] = in ? mp[i] : 0.0f;
                s.v[j] = in ? vp[i] : 0.0f;
            }
        }
    }
    if constexpr (k8) {
        s.m_scale = t.m_scale[e0 / kBlockElems];
        s.v_scale = t.v_scale[e0 / kBlockElems];
    }
}

// The update of a block, in registers.  8-bit states: m, v become the new
// bytes and scales; everything past the end of a partial block is 0 and
// leaves the block's largest values alone.
__device__ __forceinline__ void update_block(const ListTensor&, int32_t, bool, int,
                                             float (&w)[kLane], const float (&g)[kLane],
                                             Moments<false>& x, float s, const StepScalars& k,
                                             float d, uint32_t)
{
#pragma unroll
    for (int j = 0; j < kLane; ++j)
        adamwdev::adamw_elem(w[j], g[j], x.m[j], x.v[j], s, k, d);
}
__device__ __forceinline__ void update_block(const ListTensor& t, int32_t e0, bool vec, int lane,
                                             float (&w)[kLane], const float (&g)[kLane],
                                             Moments<true>& x, float s, const StepScalars& k,
                                             float d, uint32_t key)
{
    float m[kLane], v[kLane];
    float m_most = 0.0f, v_most = 0.0f;
#pragma unroll
    for (int j = 0; j < kLane; j += 2) {
        const float2 m2 = state8::widen_m((x.m[j >> 2] >> (8 * (j & 3))) & 0xffffu);
        const float2 v2 = state8::widen_v((x.v[j >> 2] >> (8 * (j & 3))) & 0xffffu);
        m[j] = __fmul_rn(m2.x, x.m_scale);
        m[j + 1] = __fmul_rn(m2.y, x.m_scale);
        v[j] = __fmul_rn(v2.x, x.v_scale);
        v[j + 1] = __fmul_rn(v2.y, x.v_scale);
    }
#pragma unroll
    for (int j = 0; j < kLane; ++j) {
        state8::moments(__fmul_rn(g[j], s), m[j], v[j], k);
        w[j] = state8::weight(w[j], m[j], v[j], k, d);
        m_most = fmaxf(m_most, fabsf(m[j]));
        v_most = fmaxf(v_most, v[j]);
    }
    // non-negative floats order as their bits do
    const uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(m_most));
    const uint32_t vb = __reduce_max_sync(0xffffffffu, __float_as_uint(v_most));
    const uint32_t me = state8::scale_exponent(mb, state8::kMTop);
    const uint32_t ve = state8::scale_exponent(vb, state8::kVTop);
    x.m_scale = state8::scale_of(me);
    x.v_scale = state8::scale_of(ve);
    const uint64_t p0 = uint64_t(t.block0) * kBlockElems + uint32_t(e0);
    const uint32_t here = key ^ (uint32_t(p0 >> 32) * 0x9E3779B1u);
    uint32_t r[kLane];
#pragma unroll
    for (int j = 0; j < kLane; ++j)
        r[j] = hash32((uint32_t(p0) + uint32_t(element(vec, lane, j))) ^ here);
    if (mb < state8::kMFast && vb < state8::kVFast) {  // the same in every lane
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            x.m[h] = state8::narrow4_m(m + 4 * h, state8::move_m(me), r + 4 * h);
            x.v[h] = state8::narrow4_v(v + 4 * h, state8::move_v(ve), r + 4 * h);
        }
    } else {
        x.m[0] = x.m[1] = x.v[0] = x.v[1] = 0u;
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            x.m[j >> 2] |= state8::narrow_m(m[j], state8::inverse_of(me), r[j]) << (8 * (j & 3));
            x.v[j >> 2] |= state8::narrow_v(v[j], state8::inverse_of(ve), r[j]) << (8 * (j & 3));
        }
    }
}

template <typename G, bool k8>
__device__ __forceinline__ void store_block(const ListTensor& t, int32_t e0, int32_t left,
                                            bool vec, int lane, const float (&w)[kLane],
                                            const Moments<k8>& s, bool zero_grad,
                                            int32_t w_lp_dtype)
{
    float* const wp = t.w + e0;
    G* const gp = static_cast<G*>(t.g) + e0;
    using State = typename std::conditional<k8, uint8_t, float>::type;
    State* const mp = static_cast<State*>(t.m) + e0;
    State* const vp = static_cast<State*>(t.v) + e0;
    if (vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = h * (kBlockElems / 2) + lane * 4;
            __stcs(reinterpret_cast<float4*>(wp + i), as_float4(w, h));
            if constexpr (k8) {
                __stcs(reinterpret_cast<uint32_t*>(mp + i), s.m[h]);
                __stcs(reinterpret_cast<uint32_t*>(vp + i), s.v[h]);
            } else {
                __stcs(reinterpret_cast<float4*>(mp + i), as_float4(s.m, h));
                __stcs(reinterpret_cast<float4*>(vp + i), as_float4(s.v, h));
            }
            if (t.w_lp && w_lp_dtype == kDtypeF16)
                detail::store4_lp_cs(static_cast<__half*>(t.w_lp) + e0 + i, as_float4(w, h));
            else if (t.w_lp)
                detail::store4_lp_cs(static_cast<__nv_bfloat16*>(t.w_lp) + e0 + i, as_float4(w, h));
            if (zero_grad)
                detail::store4_zero_cs(gp + i);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            const int i = j * 32 + lane;
            if (i >= left)
                continue;
            wp[i] = w[j];
            if constexpr (k8) {
                mp[i] = uint8_t(s.m[j >> 2] >> (8 * (j & 3)));
                vp[i] = uint8_t(s.v[j >> 2] >> (8 * (j & 3)));
            } else {
                mp[i] = s.m[j];
                vp[i] = s.v[j];
            }
            if (t.w_lp && w_lp_dtype == kDtypeF16)
                detail::store1_lp(static_cast<__half*>(t.w_lp) + e0 + i, w[j]);
            else if (t.w_lp)
                detail::store1_lp(static_cast<__nv_bfloat16*>(t.w_lp) + e0 + i, w[j]);
            if (zero_grad)
                detail::store1_zero(gp + i);
        }
    }
    if constexpr (k8) {
        if (lane == 0) {
            t.m_scale[e0 / kBlockElems] = s.m_scale;
            t.v_scale[e0 / kBlockElems] = s.v_scale;
        }
    }
}

// The update of the list's units of one kind of state.  Every block first
// adds the norm's partials up in the same fixed order (the same bits
// everywhere; block 0 of the kernel that runs first publishes the result),
// as the fused kernel of the flat state does.  The first unit's inputs are
// asked for before that: the norm kernel writes none of them.
//
// A block takes one unit after another, a warp of it one block of elements.
// While a unit is updated, the block's first warp fetches the next one's
// tensor into shared memory and draws the one after that: neither table's
// latency is waited for, and the pointers take no registers.  Long lists
// hand the units out by a counter, which keeps the blocks close to one
// another in memory.
template <typename G, bool k8>
__global__ void __launch_bounds__(kNormThreads, MINB)
    k_list_step(ListView list, StepScalars k, uint32_t key, bool publish, bool zero_grad,
                int32_t w_lp_dtype)
{
    const int lane = threadIdx.x & 31;
    const int32_t warp_e0 = int32_t(threadIdx.x >> 5) * kBlockElems;
    __shared__ ListTensor s_tensor[2];
    __shared__ int32_t s_unit[2];  // its unit, or -1: no more
    __shared__ float s_scale;
    __shared__ int s_skip;
    uint32_t* const ctr = k.chunk_ctr;
    int32_t u = int32_t(blockIdx.x);  // the unit fetched next (the first warp's)
    auto fetch = [&](int to) {
        // lane 0 draws the number of the unit after this one meanwhile
        int32_t after = u + int32_t(gridDim.x);
        if (ctr && lane == 0)
            after = int32_t(gridDim.x + atomicAdd(ctr, 1u));
        ListUnit unit{0, -1};
        if (u < list.n_units) {
            unit = list.units[u];
            constexpr int kWords = int(sizeof(ListTensor) / 16);
            if (lane < kWords)
                reinterpret_cast<uint4*>(&s_tensor[to])[lane] =
                    reinterpret_cast<const uint4*>(list.tensors + unit.tensor)[lane];
        }
        if (lane == 0)
            s_unit[to] = unit.unit;
        u = ctr ? __shfl_sync(0xffffffffu, after, 0) : after;
    };
    if (threadIdx.x < 32)
        fetch(0);
    float s = 0.0f;
    for (int i = 0;; ++i) {
        __syncthreads();
        const ListTensor& t = s_tensor[i & 1];
        const int32_t unit = s_unit[i & 1];
        const int32_t e0 = unit * kUnitElems + warp_e0;
        const int32_t left = unit < 0 ? 0 : t.numel - e0;
        const bool vec = left >= kBlockElems && (t.flags & kListVec);
        float w[kLane], g[kLane];
        Moments<k8> x;
        if (left > 0)
            load_block<G, k8>(t, e0, left, vec, lane, w, g, x);
        if (threadIdx.x < 32 && unit >= 0)
            fetch((i + 1) & 1);
        if (i == 0) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            const double total = normdev::sum_partials(k.fin.partials, k.fin.nparts);
            if (threadIdx.x == 0) {
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
        if (left > 0) {
            update_block(t, e0, vec, lane, w, g, x, s, k, (t.flags & kListDecay) ? k.decay : 1.0f,
                         key);
            store_block<G, k8>(t, e0, left, vec, lane, w, x, zero_grad, w_lp_dtype);
        }
    }
    if (ctr && threadIdx.x == 0) {
        // the last block out resets the counters for the next launch
        __threadfence();
        if (atomicAdd(ctr + 1, 1u) == gridDim.x - 1) {
            atomicExch(ctr, 0u);
            atomicExch(ctr + 1, 0u);
        }
    }
}

template <typename G, bool k8>
int launch_step_typed(const ListView& list, int32_t w_lp_dtype, const StepScalars& k,
                      uint32_t key, bool publish, bool zero_grad, int sm_count, cudaStream_t s)
{
    auto* const kernel = &k_list_step<G, k8>;
    cudaError_t err = cudaSuccess;
    static const int per_sm = detail::resident_blocks(reinterpret_cast<const void*>(kernel),
                                                      kNormThreads, 1, &err);
    const int32_t most = per_sm * sm_count;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(list.n_units < 1 ? 1 : list.n_units > most ? most : list.n_units));
    cfg.blockDim = dim3(kNormThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    StepScalars kk = k;
    if (int64_t(list.n_units) * kUnitElems < kDynamicChunksMinN)
        kk.chunk_ctr = nullptr;
    return int(cudaLaunchKernelEx(&cfg, kernel, list, kk, key, publish, zero_grad, w_lp_dtype));
}

template <typename G>
int launch_step(const ListView& plain, const ListView& eight, int32_t w_lp_dtype,
                const StepScalars& k, uint32_t key, bool zero_grad, int sm_count, cudaStream_t s)
{
    // a list without elements still publishes its norm; each kernel has its
    // own counters
    StepScalars k8 = k;
    k8.chunk_ctr = k.chunk_ctr + 2;
    int e = cudaSuccess;
    if (plain.n_units > 0 || eight.n_units == 0)
        e = launch_step_typed<G, false>(plain, w_lp_dtype, k, key, true, zero_grad, sm_count, s);
    if (e == cudaSuccess && eight.n_units > 0)
        e = launch_step_typed<G, true>(eight, w_lp_dtype, k8, key, plain.n_units == 0, zero_grad,
                                       sm_count, s);
    return e;
}

}  // namespace

int launch_list_norm(const ListView& list, int32_t g_dtype, double* partials, void* stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int blocks = list_norm_blocks(list.n_units);
    if (g_dtype == kDtypeBF16)
        k_list_norm<__nv_bfloat16><<<blocks, kNormThreads, 0, s>>>(list, partials);
    else if (g_dtype == kDtypeF16)
        k_list_norm<__half><<<blocks, kNormThreads, 0, s>>>(list, partials);
    else
        k_list_norm<float><<<blocks, kNormThreads, 0, s>>>(list, partials);
    return int(cudaGetLastError());
}

int launch_list_step(const ListView& plain, const ListView& eight, int32_t g_dtype,
                     int32_t w_lp_dtype, const StepScalars& k, uint32_t key, bool zero_grad,
                     int sm_count, void* stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (g_dtype == kDtypeBF16)
        return launch_step<__nv_bfloat16>(plain, eight, w_lp_dtype, k, key, zero_grad, sm_count, s);
    if (g_dtype == kDtypeF16)
        return launch_step<__half>(plain, eight, w_lp_dtype, k, key, zero_grad, sm_count, s);
    return launch_step<float>(plain, eight, w_lp_dtype, k, key, zero_grad, sm_count, s);
}

}  // namespace osr
