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

template <int kAct, bool kVector>
__global__ void __launch_bounds__(kSlopeThreads, 4)
    k_linear_slope(const LinearSlope a)
{
    __shared__ float sums[8][kSlopeColumns + 8];
    wait_before();
    go_ahead();
    constexpr int kAtOnce = kAct == LINEAR_NONE ? 4 : 2;
    const int lane = threadIdx.x % 32, group = threadIdx.x / 32;
    const int place = kVector ? 8 * lane : lane, step = kVector ? 1 : 32;
    const int64_t column = int64_t(blockIdx.x) * kSlopeColumns + place;
    const int64_t left = a.columns - column;
    const int count = left <= 0 ? 0 : int(left >= 8 * step ? 8 : (left + step - 1) / step);
    const int64_t first = a.rows * blockIdx.y / a.strips;
    const int64_t last = a.rows * (blockIdx.y + 1) / a.strips;
    const uint16_t* dy = static_cast<const uint16_t*>(a.dy) + (first + group) * a.dy_stride + column;
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
    const int64_t mine = int64_t(blockIdx.x) * kSlopeColumns + threadIdx.x;
    if (mine < a.columns) {
        float s = 0.0f;
#pragma unroll
        for (int g = 0; g < 8; ++g)
            s += sums[g][threadIdx.x];
        a.partials[blockIdx.y * a.columns + mine] = s;
    }
}

// dbias from the strips' sums: a block has 32 columns, a warp every 32nd strip
// of them, then a column, whose 32 sums it joins.
constexpr int kBiasThreads = 1024;
__global__ void __launch_bounds__(kBiasThreads)
    k_linear_bias_grad(const float* partials, int32_t strips, int64_t columns, void* dbias,
                       int32_t dtype, bool accumulate)
{
    __shared__ float sums[32][33];
    wait_before();
    go_ahead();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t base = int64_t(blockIdx.x) * 32;
    float s = 0.0f;
    if (base + lane < columns)
#pragma unroll 4
        for (int32_t i = warp; i < strips; i += 32)
            s += __ldcg(partials + i * columns + base + lane);
    sums[warp][lane] = s;
    __syncthreads();
    s = sums[lane][warp];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    const int64_t column = base + warp;
    if (lane == 0 && column < columns)
        store_as(dbias, column, dtype, accumulate ? s + load_as(dbias, column, dtype) : s);
}

constexpr int kCopyThreads = 256;
__global__ void __launch_bounds__(kCopyThreads)
    k_copy_rows(const uint16_t* from, int64_t from_stride, uint16_t* to, int64_t to_stride,
                int64_t rows, int64_t columns)
{
    wait_before();
    go_ahead();
    const int64_t vectors = (columns + 7) / 8;
    for (int64_t i = int64_t(blockIdx.x) * kCopyThreads + threadIdx.x; i < rows * vectors;
         i += int64_t(gridDim.x) * kCopyThreads) {
        const int64_t r = i / vectors, c = (i - r * vectors) * 8;
        const uint16_t* const p = from + r * from_stride + c;
        const int count = int(columns - c < 8 ? columns - c : 8);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = 2 * j < count ? p[2 * j] : 0u;
            const uint32_t hi = 2 * j + 1 < count ? p[2 * j + 1] : 0u;
            w[j] = lo | (hi << 16);
        }
        *reinterpret_cast<uint4*>(to + r * to_stride + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
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
    const dim3 grid(unsigned((a.columns + kSlopeColumns - 1) / kSlopeColumns), unsigned(a.strips));
    const auto on_vector = [](const void* p, int64_t stride) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0;
    };
    const bool vector = on_vector(a.dy, a.rows > 1 ? a.dy_stride : 0) &&
                        (a.act == LINEAR_NONE || on_vector(a.z, a.rows > 1 ? a.z_stride : 0));
    const auto launch = [&](void (*vectors)(LinearSlope), void (*others)(LinearSlope)) {
        return launch_early(vector ? vectors : others, grid, kSlopeThreads, 0,
                            static_cast<cudaStream_t>(stream), a);
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

int launch_linear_bias_grad(const float* partials, int32_t strips, int64_t columns, void* dbias,
                            int32_t dtype, bool accumulate, void* stream)
{
    return launch_early(k_linear_bias_grad, dim3(unsigned((columns + 31) / 32)), kBiasThreads, 0,
                        static_cast<cudaStream_t>(stream), partials, strips, columns, dbias, dtype,
                        accumulate);
}

int launch_copy_rows(const void* from, int64_t from_stride, void* to, int64_t to_stride,
                     int64_t rows, int64_t columns, void* stream)
{
    const int64_t want = (rows * ((columns + 7) / 8) + kCopyThreads - 1) / kCopyThreads;
    return launch_early(k_copy_rows, dim3(unsigned(want < 4096 ? want : 4096)), kCopyThreads, 0,
                        static_cast<cudaStream_t>(stream), static_cast<const uint16_t*>(from),
                        from_stride, static_cast<uint16_t*>(to), to_stride, rows, columns);
}

}  // namespace osr
