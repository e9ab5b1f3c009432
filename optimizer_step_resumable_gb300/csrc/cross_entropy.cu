// cross_entropy.cu -- loss and gradient of a softmax over a large vocabulary.
//
// Logits are 2 vocab dim operations a row and never leave the tensor memory:
// the epilogue of each tile turns 256 of them a row into a maximum and a sum
// of exponentials (forward), or into the logits' gradient, in 16 bits, for a
// piece of the vocabulary (backward).  In powers of two: with l' = l log2 e,
// a row's m = max l' and s = sum 2^(l' - m) give lse = (m + log2 s) ln 2; the
// rounding of m cancels.
#include <cmath>

#include "cross_entropy.h"
#include "linear_gemm.cuh"

namespace osr {
namespace {

using namespace detail;

constexpr float kLn2 = 0.69314718055994531f;

// What exponentials are taken relative to: never -inf, of which the
// difference to itself is no number.
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.0f : m; }

// v[i], bit by bit of i: a chain of comparisons becomes a place in memory, and
// with it all of v.
template <int C>
__device__ __forceinline__ float pick(const float (&v)[C], int32_t i)
{
    if constexpr (C == 1) {
        return v[0];
    } else {
        float half[C / 2];
#pragma unroll
        for (int j = 0; j < C / 2; ++j)
            half[j] = i & (C / 2) ? v[j + C / 2] : v[j];
        return pick(half, i & (C / 2 - 1));
    }
}

struct PartsEpilogue {
    static constexpr int kUnroll = 2;
    struct Params {
        const int64_t* target;
        float2* parts;
        float* at;
    };
    int32_t row, part;
    int64_t target;
    float most = -INFINITY, sum = 0.0f;  // most in units of the logits

    __device__ PartsEpilogue(const Params& p, const GemmShape& s, int32_t r, int32_t, int32_t,
                             const GemmItem& it, int32_t half, float*)
        : row(r), part(it.tile_n * kCeParts + half), target(r < s.m ? p.target[r] : -1)
    {
    }
    template <int C>
    __device__ __forceinline__ void chunk(const Params& p, const GemmShape& s, int32_t column, int,
                                          float (&v)[C], float*)
    {
        if (column >= s.n)
            return;
        if (column + C > s.n)
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (column + i >= s.n)
                    v[i] = -INFINITY;
        const int64_t off = target - column;
        if (off >= 0 && off < C && row < s.m && target < s.n)
            p.at[row] = pick(v, int32_t(off));
        float top[4] = {fmaxf(most, v[0]), v[1], v[2], v[3]};
#pragma unroll
        for (int i = 4; i < C; ++i)
            top[i % 4] = fmaxf(top[i % 4], v[i]);
        const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        const float base = reference(now) * kLog2E;
        float2 add[2] = {make_float2(sum * exp2_fast(fmaf(most, kLog2E, -base)), 0.0f),
                         make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int i = 0; i < C; i += 2)
            add[i / 2 % 2] = packed::add2(
                add[i / 2 % 2],
                exp2_fast(packed::fma2(make_float2(v[i], v[i + 1]), packed::both(kLog2E),
                                       packed::both(-base))));
        sum = (add[0].x + add[1].x) + (add[0].y + add[1].y);
        most = now;
    }
    __device__ void end(const Params& p, const GemmShape& s)
    {
        if (row < s.m)
            p.parts[int64_t(part) * s.m + row] = make_float2(reference(most) * kLog2E, sum);
    }
};

// A block joins the parts of 32 rows: eight threads a row, each every eighth.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) k_ce_join(const CeJoin a)
{
    __shared__ float2 part[8][32];
    wait_before();
    go_ahead();
    const int lane = threadIdx.x % 32, group = threadIdx.x / 32;
    const int64_t row = int64_t(blockIdx.x) * 32 + lane;
    float most = -INFINITY, sum = 0.0f;
    if (row < a.rows)
#pragma unroll 8
        for (int32_t i = group; i < a.count; i += 8) {
            const float2 p = __ldcg(a.parts + i * a.rows + row);
            // a part without columns has the sum 0, whatever its maximum
            const float now = p.y == 0.0f ? most : fmaxf(most, p.x);
            const float base = reference(now);
            sum = sum * exp2f(most - base) + p.y * exp2f(fminf(p.x - base, 0.0f));
            most = now;
        }
    part[group][lane] = make_float2(reference(most), sum);
    __syncthreads();
    if (group > 0 || row >= a.rows)
        return;
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < 8; ++g)
        top = part[g][lane].y == 0.0f ? top : fmaxf(top, part[g][lane].x);
    const float base = reference(top);
    float total = 0.0f;
#pragma unroll
    for (int g = 0; g < 8; ++g)
        total += part[g][lane].y * exp2f(fminf(part[g][lane].x - base, 0.0f));
    const float lse = (base + log2f(total)) * kLn2;
    if (a.lse)
        a.lse[row] = lse;
    const int64_t t = a.target[row];
    a.loss[row] = t < 0          ? 0.0f
                  : t >= a.vocab ? NAN
                                 : lse - a.at[row] + a.z_loss * lse * lse;
}

// What the gradient of a row's logits is made of: dloss (1 + 2 z lse) and dloss.
// The scale of all rows is left to the products' epilogues: here its bits would
// meet the rounding to 16 bits, and the targets' places, all near minus the same
// number, would err alike (1001 x 509 x 10007 binary16 gradients: 4.8e-4 off so,
// 2.2e-4 as it is).
__device__ __forceinline__ float2 factors(const CeFactors& f, int64_t row, int64_t target,
                                          float lse)
{
    if (target < 0)
        return make_float2(0.0f, 0.0f);
    if (target >= f.vocab)
        return make_float2(NAN, NAN);
    const float g = f.dloss ? f.dloss[row] : 1.0f;
    return make_float2(g * fmaf(f.two_z, lse, 1.0f), g);
}

// One block: the power of two that brings the largest that a row's gradient of a
// logit can be to [2^14, 2^15), and its inverse: p factor.x, and at the target
// p factor.x - factor.y, for any p from 0 to 1.  Binary16 ends at 65504 and loses
// bits below 2^-14.
constexpr int kCeNormThreads = 1024;
__global__ void __launch_bounds__(kCeNormThreads) k_ce_norm(const CeFactors f, int64_t rows,
                                                          float* norms)
{
    __shared__ float largest[32];
    wait_before();
    go_ahead();
    float most = 0.0f;
#pragma unroll 4
    for (int64_t r = threadIdx.x; r < rows; r += kCeNormThreads) {
        const float2 g = factors(f, r, f.target[r], f.lse[r]);
        most = fmaxf(most, fmaxf(fmaxf(fabsf(g.x), fabsf(g.y)), fabsf(g.x - g.y)));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, off));
    if (threadIdx.x % 32 == 0)
        largest[threadIdx.x / 32] = most;
    __syncthreads();
    if (threadIdx.x > 0)
        return;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        most = fmaxf(most, largest[i]);
    int shift = 0;
    if (most > 0.0f && most < INFINITY)
        shift = min(max(14 - (int(__float_as_uint(most) >> 23) - 127), -100), 100);
    norms[0] = __uint_as_float(uint32_t(127 + shift) << 23);
    norms[1] = __uint_as_float(uint32_t(127 - shift) << 23);
}

// p factor.x is 2^(l' - lse' + log2 |factor.x|), with factor.x's sign put on
// the rounded values: no product an element.
template <bool kBf16>
struct GradientEpilogue {
    static constexpr int kUnroll = 4;
    struct Params {
        CeFactors f;
        uint16_t* gradient;
        int64_t stride;
        int32_t first;
    };
    int32_t row;
    bool counts;
    int64_t target;  // in the piece
    float base, minus;
    uint32_t sign;

    __device__ GradientEpilogue(const Params& p, const GemmShape& s, int32_t r, int32_t, int32_t,
                                const GemmItem&, int32_t, float*)
        : row(r), counts(false), target(-1), base(0.0f), minus(0.0f), sign(0)
    {
        if (r >= s.m)
            return;
        const int64_t t = p.f.target[r];
        const float lse = p.f.lse[r], norm = p.f.norm ? *p.f.norm : 1.0f;
        const float2 raw = factors(p.f, r, t, lse);
        const float2 factor = make_float2(raw.x * norm, raw.y * norm);
        counts = t >= 0;
        base = log2f(fabsf(factor.x)) - lse * kLog2E;
        minus = factor.y;
        sign = factor.x < 0.0f ? 0x80008000u : 0u;
        target = t - p.first;
    }
    template <int C>
    __device__ __forceinline__ void chunk(const Params& p, const GemmShape& s, int32_t column,
                                          int c, float (&v)[C], float* stage)
    {
        const int64_t off = target - column;
        const bool here = off >= 0 && off < C && counts;
        uint32_t w[C / 2];
#pragma unroll
        for (int i = 0; i < C; i += 2) {
            const float2 e = exp2_fast(packed::fma2(make_float2(v[i], v[i + 1]),
                                                    packed::both(kLog2E), packed::both(base)));
            v[i] = e.x, v[i + 1] = e.y;
            w[i / 2] = narrow32(e.x, e.y, kBf16) ^ sign;
        }
        if (here) {
            // the target's place anew
            const float e = pick(v, int32_t(off)), at = (sign ? -e : e) - minus;
            const uint32_t half = narrow16(at, kBf16);
#pragma unroll
            for (int i = 0; i < C / 2; ++i) {
                w[i] = int32_t(off) == 2 * i ? (w[i] & 0xFFFF0000u) | half : w[i];
                w[i] = int32_t(off) == 2 * i + 1 ? (w[i] & 0xFFFFu) | (half << 16) : w[i];
            }
        }
        if (!counts)  // whatever its logits
#pragma unroll
            for (int i = 0; i < C / 2; ++i)
                w[i] = 0;
        uint4* const strip = reinterpret_cast<uint4*>(stage);
#pragma unroll
        for (int i = 0; i < C / 8; ++i)
            strip_put(strip, (c & 1) * (C / 8) + i,
                      make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
        if (c & 1) {  // whole tiles fit the rows of the gradient
            const int32_t first = row - int32_t(threadIdx.x % 32);
            strip_write(strip, p.gradient + first * p.stride + column - C, p.stride, s.m - first,
                        2 * C);
        }
    }
    __device__ void end(const Params&, const GemmShape&) {}
};

template <typename E>
int run(const GemmOperand& x, const GemmOperand& weight, bool bf16, const typename E::Params& p,
        int sm_count, int32_t* gave_up, void* stream)
{
    GemmShape s{};
    s.splits = s.chains = 1;
    s.gave_up = gave_up;
    return gemm_run<kCeColumns, E>(x, weight, s, bf16, p, GemmSide{}, sm_count,
                                   static_cast<cudaStream_t>(stream));
}

}  // namespace

int launch_ce_parts(const CeForward& a, int sm_count, int32_t* gave_up, void* stream)
{
    return run<PartsEpilogue>(a.x, a.weight, a.bf16, {a.target, a.parts, a.at}, sm_count, gave_up,
                              stream);
}

int launch_ce_join(const CeJoin& a, void* stream)
{
    return launch_early(k_ce_join, dim3(unsigned((a.rows + 31) / 32)), kJoinThreads, 0,
                        static_cast<cudaStream_t>(stream), a);
}

int launch_ce_norm(const CeFactors& f, int64_t rows, float* norms, void* stream)
{
    return launch_early(k_ce_norm, dim3(1), kCeNormThreads, 0, static_cast<cudaStream_t>(stream), f,
                        rows, norms);
}

int launch_ce_gradient(const CeGradient& a, int sm_count, int32_t* gave_up, void* stream)
{
    const auto launch = [&](auto epilogue) {
        using E = decltype(epilogue);
        return run<std::remove_pointer_t<E>>(
            a.x, a.weight, a.bf16,
            {a.factors, static_cast<uint16_t*>(a.gradient), a.stride, a.first},
            sm_count, gave_up, stream);
    };
    return a.bf16 ? launch(static_cast<GradientEpilogue<true>*>(nullptr))
                  : launch(static_cast<GradientEpilogue<false>*>(nullptr));
}

}  // namespace osr
