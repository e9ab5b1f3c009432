// linear_rows.cu -- the linear layer's passes over rows: the gradient through
// the activation with the bias's gradient, and copies of rows that the tiled
// copies cannot read.  All are bound by memory: each value is read once.
#include "early_dev.cuh"
#include "linear_dev.cuh"

namespace osr {
namespace {

using namespace detail;

// A block has 256 neighbouring columns of a strip of the rows, a warp every
// eighth row, a thread eight columns: neighbours in one vector, or, where
// rows do not start on vectors, every 32nd.  kAtOnce rows of a thread are on
// their way at a time.  The eight warps' sums of a column meet in shared
// memory.
constexpr int kSlopeThreads = 256, kSlopeColumns = 256;

__device__ __forceinline__ void widen8(uint4 q, bool bf16, float (&v)[8])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = widen16(w[i] & 0xFFFFu, bf16);
        v[2 * i + 1] = widen16(w[i] >> 16, bf16);
    }
}
// Eight elements of a row from p; `step` apart, those before `count` of them.
template <bool kVector>
__device__ __forceinline__ uint4 load8(const uint16_t* p, int step, int count)
{
    if (kVector && count >= 8)
        return __ldcs(reinterpret_cast<const uint4*>(p));
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = i < count ? p[i * step] : 0u;
    return make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16),
                      w[6] | (w[7] << 16));
}

// Copies: eight elements a thread, wherever the rows start.
__device__ __forceinline__ void copy_rows(const LinearCopy& c, int64_t block, int64_t blocks)
{
    const int64_t vectors = (c.columns + 7) / 8;
    for (int64_t i = block * blockDim.x + threadIdx.x; i < c.rows * vectors;
         i += blocks * blockDim.x) {
        const int64_t r = i / vectors, at = (i - r * vectors) * 8;
        const uint16_t* const p = static_cast<const uint16_t*>(c.from) + r * c.from_stride + at;
        const int count = int(c.columns - at < 8 ? c.columns - at : 8);
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w[j] = j < count ? p[j] : 0u;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.to) + r * c.to_stride + at) =
            make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16),
                       w[6] | (w[7] << 16));
    }
}
constexpr int kCopyThreads = 256;
int copy_blocks(const LinearCopy& c)
{
    if (!c.to)
        return 0;
    const int64_t want = (c.rows * ((c.columns + 7) / 8) + kCopyThreads - 1) / kCopyThreads;
    return int(want < 2048 ? want : 2048);
}
__global__ void __launch_bounds__(kCopyThreads)
    k_linear_copies(const LinearCopy a, const LinearCopy b, int32_t a_blocks)
{
    wait_before();
    go_ahead();
    if (int32_t(blockIdx.x) < a_blocks)
        copy_rows(a, blockIdx.x, a_blocks);
    else
        copy_rows(b, blockIdx.x - a_blocks, gridDim.x - a_blocks);
}

template <int kAct, bool kVector>
__global__ void __launch_bounds__(kSlopeThreads, 4)
    k_linear_slope(const LinearSlope a, int32_t across, int32_t copies0, int32_t copies1)
{
    __shared__ float sums[8][kSlopeColumns + 8];
    wait_before();
    go_ahead();
    // the blocks behind the strips' copy
    const int32_t copier = int32_t(blockIdx.x) - across * a.strips;
    if (copier >= 0) {
        if (copier < copies0)
            copy_rows(a.copies[0], copier, copies0);
        else
            copy_rows(a.copies[1], copier - copies0, copies1);
        return;
    }
    const int32_t strip = int32_t(blockIdx.x) / across, part = int32_t(blockIdx.x) % across;
    constexpr int kAtOnce = kAct == LINEAR_NONE ? 4 : 2;
    const int lane = threadIdx.x % 32, group = threadIdx.x / 32;
    const int place = kVector ? 8 * lane : lane, step = kVector ? 1 : 32;
    const int64_t column = int64_t(part) * kSlopeColumns + place;
    const int64_t left = a.columns - column;
    const int count = left <= 0 ? 0 : int(left >= 8 * step ? 8 : (left + step - 1) / step);
    const int64_t first = a.rows * strip / a.strips;
    const int64_t last = a.rows * (strip + 1) / a.strips;
    const uint16_t* dy =
        static_cast<const uint16_t*>(a.dy) + (first + group) * a.dy_stride + column;
    const uint16_t* z = static_cast<const uint16_t*>(a.z) + (first + group) * a.z_stride + column;
    uint16_t* dz = static_cast<uint16_t*>(a.dz) + (first + group) * a.stride + column;
    float total[8] = {};
    for (int64_t r = first + group; r < last && count > 0; r += 8 * kAtOnce) {
        uint4 g[kAtOnce], x[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (r + 8 * k < last) {
                g[k] = load8<kVector>(dy + 8 * k * a.dy_stride, step, count);
                if constexpr (kAct != LINEAR_NONE)
                    x[k] = load8<kVector>(z + 8 * k * a.z_stride, step, count);
            }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (r + 8 * k < last) {
                float f[8];
                widen8(g[k], a.bf16, f);
                if constexpr (kAct != LINEAR_NONE) {
                    float s[8];
                    widen8(x[k], a.bf16, s);
                    times_slopes<kAct>(f, s);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    total[i] += f[i];
                if (a.dz) {
                    uint16_t* const to = dz + 8 * k * a.stride;
                    if constexpr (kVector) {  // the stride is a multiple of eight
                        *reinterpret_cast<uint4*>(to) =
                            make_uint4(narrow32(f[0], f[1], a.bf16), narrow32(f[2], f[3], a.bf16),
                                       narrow32(f[4], f[5], a.bf16), narrow32(f[6], f[7], a.bf16));
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (i < count)
                                to[i * step] = narrow16(f[i], a.bf16);
                    }
                }
            }
        dy += 8 * kAtOnce * a.dy_stride;
        z += 8 * kAtOnce * a.z_stride;
        dz += 8 * kAtOnce * a.stride;
    }
    if (!a.partials)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sums[group][place + i * step] = total[i];
    __syncthreads();
    const int64_t mine = int64_t(part) * kSlopeColumns + threadIdx.x;
    if (mine < a.columns) {
        float s = 0.0f;
#pragma unroll
        for (int g = 0; g < 8; ++g)
            s += sums[g][threadIdx.x];
        a.partials[strip * a.columns + mine] = s;
    }
}

// dbias from the strips' sums: a block has 32 columns, a warp every 32nd strip
// of them, then a column, whose 32 sums it joins.
constexpr int kBiasThreads = 1024;
__global__ void __launch_bounds__(kBiasThreads)
    k_linear_bias_grad(const GemmSide s)
{
    __shared__ float sums[32][33];
    wait_before();
    go_ahead();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t base = int64_t(blockIdx.x) * 32;
    float sum = 0.0f;
    if (base + lane < s.columns)
#pragma unroll 4
        for (int32_t i = warp; i < s.strips; i += 32)
            sum += __ldcg(s.partials + i * s.columns + base + lane);
    sums[warp][lane] = sum;
    __syncthreads();
    sum = sums[lane][warp];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
    const int64_t column = base + warp;
    if (lane == 0 && column < s.columns)
        store_as(s.out, column, s.dtype, s.add ? sum + load_as(s.out, column, s.dtype) : sum);
}

}  // namespace

int linear_strips(int64_t rows, int64_t columns, int sm_count)
{
    const int64_t across = (columns + kSlopeColumns - 1) / kSlopeColumns;
    int64_t strips = (int64_t(sm_count) * 4 + across - 1) / across;
    const int64_t most = (rows + 31) / 32;  // four rows a thread at least
    strips = strips < most ? strips : most;
    strips = strips < 128 ? strips : 128;
    return int(strips > 1 ? strips : 1);
}

int launch_linear_slope(const LinearSlope& a, void* stream)
{
    const int32_t across = int32_t((a.columns + kSlopeColumns - 1) / kSlopeColumns);
    const int32_t copies[] = {copy_blocks(a.copies[0]), copy_blocks(a.copies[1])};
    const dim3 grid(unsigned(across * a.strips + copies[0] + copies[1]));
    const auto on_vector = [](const void* p, int64_t stride) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0;
    };
    const bool vector = on_vector(a.dy, a.rows > 1 ? a.dy_stride : 0) &&
                        (a.act == LINEAR_NONE || on_vector(a.z, a.rows > 1 ? a.z_stride : 0));
    using Kernel = void (*)(LinearSlope, int32_t, int32_t, int32_t);
    const auto launch = [&](Kernel vectors, Kernel others) {
        return launch_early(vector ? vectors : others, grid, kSlopeThreads, 0,
                            static_cast<cudaStream_t>(stream), a, across, copies[0], copies[1]);
    };
    switch (a.act) {
    case LINEAR_RELU:
        return launch(k_linear_slope<LINEAR_RELU, true>, k_linear_slope<LINEAR_RELU, false>);
    case LINEAR_GELU:
        return launch(k_linear_slope<LINEAR_GELU, true>, k_linear_slope<LINEAR_GELU, false>);
    case LINEAR_GELU_TANH:
        return launch(k_linear_slope<LINEAR_GELU_TANH, true>,
                      k_linear_slope<LINEAR_GELU_TANH, false>);
    case LINEAR_SILU:
        return launch(k_linear_slope<LINEAR_SILU, true>, k_linear_slope<LINEAR_SILU, false>);
    default: return launch(k_linear_slope<LINEAR_NONE, true>, k_linear_slope<LINEAR_NONE, false>);
    }
}

int launch_linear_bias_grad(const GemmSide& side, void* stream)
{
    return launch_early(k_linear_bias_grad, dim3(unsigned((side.columns + 31) / 32)), kBiasThreads,
                        0, static_cast<cudaStream_t>(stream), side);
}

int launch_linear_copies(const LinearCopy& a, const LinearCopy& b, void* stream)
{
    const int32_t a_blocks = copy_blocks(a);
    return launch_early(k_linear_copies, dim3(unsigned(a_blocks + copy_blocks(b))), kCopyThreads, 0,
                        static_cast<cudaStream_t>(stream), a, b, a_blocks);
}

}  // namespace osr
