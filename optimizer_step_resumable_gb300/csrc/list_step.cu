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

#include <cuda_runtime.h>

#include "adamw_dev.cuh"
#include "common.cuh"
#include "list.h"
#include "norm_dev.cuh"
#include "state8_dev.cuh"

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

// A lane's gradient elements of one block of `left` elements.
template <typename G>
__device__ __forceinline__ void load_g(const G* g, bool vec, int lane, int64_t left,
                                       float (&x)[kLane])
{
    if (vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 a = detail::load4_cg<G>(g + h * (kBlockElems / 2) + lane * 4);
            x[4 * h] = a.x;
            x[4 * h + 1] = a.y;
            x[4 * h + 2] = a.z;
            x[4 * h + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            const int i = j * 32 + lane;
            x[j] = i < left ? detail::load1(g + i) : 0.0f;
        }
    }
}

// Level 1 of the norm: block b's warps take units b * kWarps + warp, + the
// grid's warps, ...; a lane's share of a unit is one run of squares
// (normdev::run_sumsq), added up in double.
template <typename G>
__global__ void __launch_bounds__(kNormThreads, 4)
    k_list_norm(ListView list, double* __restrict__ partials)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    double acc = 0.0;
    for (int64_t u = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < list.n_units;
         u += int64_t(gridDim.x) * kWarps) {
        const ListUnit unit = list.units[u];
        const ListTensor& t = list.tensors[unit.tensor];
        const int64_t e0 = int64_t(unit.unit) * kUnitElems;
        const G* g = static_cast<const G*>(t.g) + e0;
        const int64_t left = t.numel - e0;
        const bool aligned = t.flags & kListVec;
        float4 x[2 * kUnitBlocks];
#pragma unroll
        for (int b = 0; b < kUnitBlocks; ++b) {
            float y[kLane];
            load_g<G>(g + b * kBlockElems, aligned && left >= (b + 1) * kBlockElems, lane,
                      left - b * kBlockElems, y);
            x[2 * b] = make_float4(y[0], y[1], y[2], y[3]);
            x[2 * b + 1] = make_float4(y[4], y[5], y[6], y[7]);
        }
        acc += normdev::run_sumsq<2 * kUnitBlocks>(x);
    }
    acc = detail::block_sum<kNormThreads>(acc);
    if (threadIdx.x == 0)
        partials[blockIdx.x] = acc;
}

// A lane's elements of a float array of one block.
__device__ __forceinline__ void load_f32(const float* p, bool vec, int lane, int64_t left,
                                         float (&x)[kLane])
{
    if (vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 a =
                __ldcs(reinterpret_cast<const float4*>(p + h * (kBlockElems / 2) + lane * 4));
            x[4 * h] = a.x;
            x[4 * h + 1] = a.y;
            x[4 * h + 2] = a.z;
            x[4 * h + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            const int i = j * 32 + lane;
            x[j] = i < left ? p[i] : 0.0f;
        }
    }
}
__device__ __forceinline__ void store_f32(float* p, bool vec, int lane, int64_t left,
                                          const float (&x)[kLane])
{
    if (vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            __stcs(reinterpret_cast<float4*>(p + h * (kBlockElems / 2) + lane * 4),
                   make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]));
    } else {
#pragma unroll
        for (int j = 0; j < kLane; ++j)
            if (j * 32 + lane < left)
                p[j * 32 + lane] = x[j];
    }
}

// A lane's bytes of a block, in two words.
__device__ __forceinline__ void load_u8(const uint8_t* p, bool vec, int lane, int64_t left,
                                        uint32_t (&c)[2])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (vec) {
            c[h] = __ldcs(reinterpret_cast<const uint32_t*>(p + h * (kBlockElems / 2) + lane * 4));
        } else {
            c[h] = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = (4 * h + j) * 32 + lane;
                if (i < left)
                    c[h] |= uint32_t(p[i]) << (8 * j);
            }
        }
    }
}
__device__ __forceinline__ void store_u8(uint8_t* p, bool vec, int lane, int64_t left,
                                         const uint32_t (&c)[2])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (vec) {
            __stcs(reinterpret_cast<uint32_t*>(p + h * (kBlockElems / 2) + lane * 4), c[h]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = (4 * h + j) * 32 + lane;
                if (i < left)
                    p[i] = uint8_t(c[h] >> (8 * j));
            }
        }
    }
}

template <typename L>
__device__ __forceinline__ void store_copy(L* p, bool vec, int lane, int64_t left,
                                           const float (&x)[kLane])
{
    if (vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            detail::store4_lp_cs(p + h * (kBlockElems / 2) + lane * 4,
                                 make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]));
    } else {
#pragma unroll
        for (int j = 0; j < kLane; ++j)
            if (j * 32 + lane < left)
                detail::store1_lp(p + j * 32 + lane, x[j]);
    }
}

template <typename G>
__device__ __forceinline__ void store_zero(G* p, bool vec, int lane, int64_t left)
{
    if (vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            detail::store4_zero_cs(p + h * (kBlockElems / 2) + lane * 4);
    } else {
#pragma unroll
        for (int j = 0; j < kLane; ++j)
            if (j * 32 + lane < left)
                detail::store1_zero(p + j * 32 + lane);
    }
}

// One block of a tensor by one warp.  e0: its first element; a partial block
// reads zeros past the end, which leave the block's largest values alone.
template <typename G>
__device__ __forceinline__ void update_block(const ListTensor& t, int64_t e0, int lane, float s,
                                             const StepScalars& k, uint32_t key, bool zero_grad,
                                             int32_t w_lp_dtype)
{
    const int64_t left = t.numel - e0;
    const bool vec = (t.flags & kListVec) && left >= kBlockElems;
    const float d = (t.flags & kListDecay) ? k.decay : 1.0f;
    G* const gp = static_cast<G*>(t.g) + e0;
    float w[kLane], g[kLane];
    load_f32(t.w + e0, vec, lane, left, w);
    load_g<G>(gp, vec, lane, left, g);
    if (t.flags & kListState8) {
        uint8_t* const mp = static_cast<uint8_t*>(t.m) + e0;
        uint8_t* const vp = static_cast<uint8_t*>(t.v) + e0;
        const int64_t b = e0 / kBlockElems;
        uint32_t mc[2], vc[2];
        load_u8(mp, vec, lane, left, mc);
        load_u8(vp, vec, lane, left, vc);
        const float ms = t.m_scale[b], vs = t.v_scale[b];
        float m[kLane], v[kLane];
        float m_most = 0.0f, v_most = 0.0f;
#pragma unroll
        for (int j = 0; j < kLane; j += 2) {
            const float2 m2 = state8::widen_m((mc[j >> 2] >> (8 * (j & 3))) & 0xffffu);
            const float2 v2 = state8::widen_v((vc[j >> 2] >> (8 * (j & 3))) & 0xffffu);
            m[j] = __fmul_rn(m2.x, ms);
            m[j + 1] = __fmul_rn(m2.y, ms);
            v[j] = __fmul_rn(v2.x, vs);
            v[j + 1] = __fmul_rn(v2.y, vs);
        }
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            state8::moments(__fmul_rn(g[j], s), m[j], v[j], k);
            w[j] = state8::weight(w[j], m[j], v[j], k, d);
            m_most = fmaxf(m_most, fabsf(m[j]));
            v_most = fmaxf(v_most, v[j]);
        }
        // non-negative floats order as their bits do
        const uint32_t me = state8::scale_exponent(
            __reduce_max_sync(0xffffffffu, __float_as_uint(m_most)), state8::kMTop);
        const uint32_t ve = state8::scale_exponent(
            __reduce_max_sync(0xffffffffu, __float_as_uint(v_most)), state8::kVTop);
        const float mi = state8::inverse_of(me), vi = state8::inverse_of(ve);
        const uint64_t p0 = (uint64_t(t.block0) + uint64_t(b)) * kBlockElems;
        const uint32_t here = key ^ (uint32_t(p0 >> 32) * 0x9E3779B1u);
        mc[0] = mc[1] = vc[0] = vc[1] = 0u;
#pragma unroll
        for (int j = 0; j < kLane; ++j) {
            const uint32_t r = hash32((uint32_t(p0) + uint32_t(element(vec, lane, j))) ^ here);
            mc[j >> 2] |= state8::narrow_m(m[j], mi, r) << (8 * (j & 3));
            vc[j >> 2] |= state8::narrow_v(v[j], vi, r) << (8 * (j & 3));
        }
        store_u8(mp, vec, lane, left, mc);
        store_u8(vp, vec, lane, left, vc);
        if (lane == 0) {
            t.m_scale[b] = state8::scale_of(me);
            t.v_scale[b] = state8::scale_of(ve);
        }
    } else {
        float* const mp = static_cast<float*>(t.m) + e0;
        float* const vp = static_cast<float*>(t.v) + e0;
        float m[kLane], v[kLane];
        load_f32(mp, vec, lane, left, m);
        load_f32(vp, vec, lane, left, v);
#pragma unroll
        for (int j = 0; j < kLane; ++j)
            adamwdev::adamw_elem(w[j], g[j], m[j], v[j], s, k, d);
        store_f32(mp, vec, lane, left, m);
        store_f32(vp, vec, lane, left, v);
    }
    store_f32(t.w + e0, vec, lane, left, w);
    if (t.w_lp) {
        if (w_lp_dtype == kDtypeF16)
            store_copy(static_cast<__half*>(t.w_lp) + e0, vec, lane, left, w);
        else
            store_copy(static_cast<__nv_bfloat16*>(t.w_lp) + e0, vec, lane, left, w);
    }
    if (zero_grad)
        store_zero<G>(gp, vec, lane, left);
}

// The update.  Every block first adds the norm's partials up in the same
// fixed order (the same bits everywhere; block 0 publishes the result), as
// the fused kernel of the flat state does.
template <typename G>
__global__ void __launch_bounds__(kNormThreads, 4)
    k_list_step(ListView list, StepScalars k, uint32_t key, bool zero_grad, int32_t w_lp_dtype)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float s_scale;
    __shared__ int s_skip;
    const double total = normdev::sum_partials(k.fin.partials, k.fin.nparts);
    if (threadIdx.x == 0) {
        const NormResult r = normdev::make_result(
            total, k.fin.clip, k.fin.grad_scale, blockIdx.x == 0 ? k.fin.d_res->seq + 1u : 0u);
        s_scale = r.scale;
        s_skip = r.nonfinite;
        if (blockIdx.x == 0)
            normdev::publish(r, k.fin.d_res, k.fin.h_res);
    }
    __syncthreads();
    if (s_skip)
        return;
    const float s = s_scale;
    const int lane = threadIdx.x & 31;
    for (int64_t u = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < list.n_units;
         u += int64_t(gridDim.x) * kWarps) {
        const ListUnit unit = list.units[u];
        const ListTensor t = list.tensors[unit.tensor];
        const int64_t e0 = int64_t(unit.unit) * kUnitElems;
        const int64_t end = t.numel < e0 + kUnitElems ? t.numel : e0 + kUnitElems;
        for (int64_t e = e0; e < end; e += kBlockElems)
            update_block<G>(t, e, lane, s, k, key, zero_grad, w_lp_dtype);
    }
}

template <typename G>
int launch_step_typed(const ListView& list, int32_t w_lp_dtype, const StepScalars& k,
                      uint32_t key, bool zero_grad, int blocks, cudaStream_t s)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kNormThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return int(cudaLaunchKernelEx(&cfg, &k_list_step<G>, list, k, key, zero_grad, w_lp_dtype));
}

}  // namespace

int query_list_blocks(int sm_count, int* blocks_out)
{
    cudaError_t err = cudaSuccess;
    *blocks_out = detail::resident_blocks(reinterpret_cast<const void*>(&k_list_step<float>),
                                          kNormThreads, sm_count, &err);
    return int(err);
}

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

int launch_list_step(const ListView& list, int32_t g_dtype, int32_t w_lp_dtype,
                     const StepScalars& k, uint32_t key, bool zero_grad, int blocks,
                     void* stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t want = detail::ceil_div(list.n_units, kWarps);
    blocks = int(want < 1 ? 1 : want > blocks ? blocks : want);
    if (g_dtype == kDtypeBF16)
        return launch_step_typed<__nv_bfloat16>(list, w_lp_dtype, k, key, zero_grad, blocks, s);
    if (g_dtype == kDtypeF16)
        return launch_step_typed<__half>(list, w_lp_dtype, k, key, zero_grad, blocks, s);
    return launch_step_typed<float>(list, w_lp_dtype, k, key, zero_grad, blocks, s);
}

}  // namespace osr
