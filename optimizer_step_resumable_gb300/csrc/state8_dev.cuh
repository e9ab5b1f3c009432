// state8_dev.cuh -- Adam moments in 8 bits: the values, the block scales and
// the random rounding.
//
// A block is kBlockElems consecutive elements of one tensor, held by one
// warp.  m is an e4m3 value (sign, 4 exponent, 3 significand bits) and v an
// e5m2 value (5 exponent, 2 significand bits; never negative), each times
// the block's scale.  The scale is the power of two that puts the block's
// largest magnitude into [2^7, 2^8) for m and [2^14, 2^15) for v -- below
// the formats' largest finite values 448 and 57344 by at least the factor
// rounding can add -- so scaling is exact both ways and the only rounding
// is the one to the 8-bit value.  Infinities and NaNs do not count for the
// scale: they spoil no element but their own (m keeps both as NaN).  v gets
// the wider format: it ranges over the square of the gradients' range.
//
// That rounding is random, up or down to a neighbour with the value as the
// mean.  With beta2 = 0.999 one step changes v by about 0.1%, against a
// spacing of 12-25% between neighbours: rounded to nearest, v would never
// move again; rounded at random it moves rarely but right on average.  The
// random numbers are a hash of (key of the step, position), so a run is
// reproducible bit for bit.  A positive v rounds to at least the smallest
// e5m2 value: with v = 0 the update would be m / eps.
//
// The moments are formed in single IEEE roundings in a fixed order (no fused
// multiply-add), so the stored bytes follow from the formulas on any machine.
// An element takes 59 instructions: memory and instructions bind the update
// about equally (without the arithmetic, 304 instead of 327 us).
#pragma once

#include <cstdint>

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "list.h"
#include "packed_dev.cuh"

namespace osr {
namespace state8 {

using packed::both;
using packed::fma2;
using packed::mul2;

constexpr int kMTop = 7, kVTop = 14;  // exponent of a block's largest value
constexpr uint32_t kInfinity = 0x7f800000u;

// The biased binary32 exponent of the scale of a block whose largest
// magnitude has the bits `most`; at least 1, so that the scale and its
// reciprocal (biased exponent 254 - e) are normal numbers.
__device__ __forceinline__ uint32_t scale_exponent(uint32_t most, int top)
{
    const int e = int(most >> 23) - top;
    return uint32_t(e < 1 ? 1 : e);
}
__device__ __forceinline__ float scale_of(uint32_t e) { return __uint_as_float(e << 23); }
__device__ __forceinline__ float inverse_of(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// Two values of one format, widened exactly.
__device__ __forceinline__ float2 widen_m(uint32_t two)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(two), __NV_E4M3);
    return __half22float2(__half2(h));
}
__device__ __forceinline__ float2 widen_v(uint32_t two)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(two), __NV_E5M2);
    return __half22float2(__half2(h));
}

// |x| / scale moved down by the two formats' difference in exponent bias:
// the 8-bit format's subnormal range then is binary32's, so that in either
// range the bits below the last kept one are the low 20 (e4m3) or 21 (e5m2)
// bits of the word; adding a random number of that many bits and cutting
// them off rounds up with the right probability.  16 random bits are used
// (their unit is 2^-16 of the spacing).
__device__ __forceinline__ uint32_t narrow_m(float x, float inverse, uint32_t random)
{
    const float y = __fmul_rn(__fmul_rn(fabsf(x), inverse), 0x1p-120f);
    uint32_t c = (__float_as_uint(y) + ((random >> 16) << 4)) >> 20;
    c = c > 0x7fu ? 0x7fu : c;  // inf, nan: nan
    return c | ((__float_as_uint(x) >> 24) & 0x80u);
}
__device__ __forceinline__ uint32_t narrow_v(float x, float inverse, uint32_t random)
{
    const float y = __fmul_rn(__fmul_rn(x, inverse), 0x1p-112f);
    uint32_t c = (__float_as_uint(y) + ((random & 0xffffu) << 5)) >> 21;
    c = c > 0x7cu ? 0x7cu : c;  // inf stays inf
    return x != x ? 0x7fu : (c == 0u && x > 0.0f) ? 1u : c;
}

// The same bytes for four elements at once in half the instructions, for
// blocks whose scale's reciprocal and the move down are one normal number:
// largest |m| below 2^14 and largest v below 2^29 (any state but a diverging
// one).  The sum is formed 4 (e4m3) or 3 (e5m2) bits further up, in one
// integer multiply-add whose random number lies in bits 8 to 23, so that
// byte 3 of each sum is a code.
constexpr uint32_t kMFast = (127u + 14u) << 23, kVFast = (127u + 29u) << 23;
__device__ __forceinline__ float move_m(uint32_t e) { return __uint_as_float((134u - e) << 23); }
__device__ __forceinline__ float move_v(uint32_t e) { return __uint_as_float((142u - e) << 23); }

__device__ __forceinline__ uint32_t gather_byte3(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}
// The codes of x[0..4) as m and y[0..4) as v, rounded by the hashes of four
// words begun as `begun`[j].
__device__ __forceinline__ void narrow4(const float* x, float move_x, const float* y, float move_y,
                                        const uint32_t* begun, uint32_t& cx, uint32_t& cy)
{
    uint32_t s[4], z[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // hash32_end's last step, for each half in its place: the high half
        // of h ^ h >> 16 is h's, the low one the exclusive or of both
        const uint32_t h = hash32_middle(begun[j]);
        const uint32_t high = __byte_perm(h, 0u, 0x4324);
        const uint32_t low = __byte_perm(h, 0u, 0x4104) ^ high;
        s[j] = __float_as_uint(__fmul_rn(fabsf(x[j]), move_x)) * 16u + high;
        z[j] = __float_as_uint(__fmul_rn(y[j], move_y)) * 8u + low;
    }
    const uint32_t signs = gather_byte3(__float_as_uint(x[0]), __float_as_uint(x[1]),
                                        __float_as_uint(x[2]), __float_as_uint(x[3]));
    cx = gather_byte3(s[0], s[1], s[2], s[3]) | (signs & 0x80808080u);
    cy = gather_byte3(z[0], z[1], z[2], z[3]);
    if ((cy - 0x01010101u) & ~cy & 0x80808080u) {  // some code is 0
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (y[j] > 0.0f && !((cy >> (8 * j)) & 0xffu))
                cy |= 1u << (8 * j);
    }
}

// Two elements' moments (the formulas of adamw_elem, with every product and
// sum rounded on its own: packed sums would be joined with the products into
// fused multiply-adds).  b1 and b2: the betas times the block's old scales.
__device__ __forceinline__ void moments(float2 gh, float2 m_old, float2 v_old, float b1, float b2,
                                        const StepScalars& k, float* m, float* v)
{
    const float2 p = mul2(both(b1), m_old), q = mul2(both(k.omb1), gh);
    m[0] = __fadd_rn(p.x, q.x);
    m[1] = __fadd_rn(p.y, q.y);
    const float2 r = mul2(both(b2), v_old), u = mul2(mul2(both(k.omb2), gh), gh);
    v[0] = __fadd_rn(r.x, u.x);
    v[1] = __fadd_rn(r.y, u.y);
}

// Two elements' weights.  root: sqrt(v) in units of 1 / inv; the quotient to
// 2 units of 2^-23 (the denominator is 0 or a normal number): the update is a
// small part of w.
__device__ __forceinline__ float2 weight(float2 w, float2 m, float2 root, float inv,
                                         const StepScalars& k, float d)
{
    const float2 denom = fma2(root, both(inv), both(k.eps));
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(denom.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(denom.y));
    return fma2(w, both(d), mul2(both(-k.step_size), mul2(m, r)));
}
// sqrt(v) / kRootUnit for v below kVFast, to 2^-23: moved up by 2^32 first,
// so that the square root, which takes subnormal numbers for 0, meets none.
constexpr float kRootUnit = 0x1p-16f;
__device__ __forceinline__ float2 root_fast(float2 v)
{
    const float2 u = mul2(v, both(0x1p32f));
    float2 r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(u.x));
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(u.y));
    return r;
}
// NaN if one of them is.
__device__ __forceinline__ float largest(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

}  // namespace state8
}  // namespace osr
