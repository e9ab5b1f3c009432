// linear_rows.cu -- the linear layer's passes over rows: the gradient through
// the activation with the bias's gradient, and copies of rows that the tiled
// copies cannot read.  All are bound by memory: each value is read once.
#include "early_dev.cuh"
#include "linear_dev.cuh"

namespace osr {
namespace {

using namespace detail;

// A block has 256 neighbouring columns, eight a thread, and every eighth row
// of its strip a thread; the eight partial sums of a column meet in shared
// memory.
constexpr int kSlopeThreads = 256, kSlopeColumns = 256;

// Eight 16-bit values; vectors: p is on a 16-byte boundary.
__device__ __forceinline__ void load8(const uint16_t* p, int count, bool vectors, bool bf16,
                                      float (&v)[8])
{
    if (vectors && count >= 8) {
        const uint4 r = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = widen16(w[i] & 0xFFFFu, bf16);
            v[2 * i + 1] = widen16(w[i] >> 16, bf16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = i < count ? widen16(p[i], bf16) : 0.0f;
    }
}

template <int kAct>
__global__ void __launch_bounds__(kSlopeThreads) k_linear_slope(const LinearSlope a)
{
    __shared__ float sums[8][kSlopeColumns + 8];
    wait_before();
    go_ahead();
    const int lane = threadIdx.x % 32, group = threadIdx.x / 32;
    const int64_t column = int64_t(blockIdx.x) * kSlopeColumns + 8 * lane;
    const int64_t left = a.columns - column;
    const int count = int(left < 8 ? (left < 0 ? 0 : left) : 8);
    const int64_t first = a.rows * blockIdx.y / a.strips;
    const int64_t last = a.rows * (blockIdx.y + 1) / a.strips;
    const bool dy_vectors = reinterpret_cast<uintptr_t>(a.dy) % 16 == 0 && a.dy_stride % 8 == 0;
    const bool z_vectors = reinterpret_cast<uintptr_t>(a.z) % 16 == 0 && a.z_stride % 8 == 0;
    float total[8] = {};
    if (count > 0)
#pragma unroll 4
        for (int64_t r = first + group; r < last; r += 8) {
            float g[8];
            load8(static_cast<const uint16_t*>(a.dy) + r * a.dy_stride + column, count,
                  dy_vectors, a.bf16, g);
            if constexpr (kAct != LINEAR_NONE) {
                float z[8];
                load8(static_cast<const uint16_t*>(a.z) + r * a.z_stride + column, count,
                      z_vectors, a.bf16, z);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    g[i] *= slope<kAct>(z[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                total[i] += g[i];
            if (a.dz) {  // rows of whole vectors: the stride is a multiple of eight
                const uint4 w = make_uint4(
                    narrow32(g[0], g[1], a.bf16), narrow32(g[2], g[3], a.bf16),
                    narrow32(g[4], g[5], a.bf16), narrow32(g[6], g[7], a.bf16));
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dz) + r * a.stride + column) = w;
            }
        }
    if (!a.partials)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sums[group][8 * lane + i] = total[i];
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

// dbias from the strips' sums, in order: four interleaved sums a column, one
// for each quarter of the block.
constexpr int kBiasThreads = 256;
__global__ void __launch_bounds__(kBiasThreads)
    k_linear_bias_grad(const float* partials, int32_t strips, int64_t columns, void* dbias,
                       int32_t dtype, bool accumulate)
{
    __shared__ float sums[4][64];
    wait_before();
    go_ahead();
    const int lane = threadIdx.x % 64, part = threadIdx.x / 64;
    const int64_t column = int64_t(blockIdx.x) * 64 + lane;
    float s = 0.0f;
    if (column < columns)
#pragma unroll 8
        for (int32_t i = part; i < strips; i += 4)
            s += __ldcg(partials + i * columns + column);
    sums[part][lane] = s;
    __syncthreads();
    if (part == 0 && column < columns) {
        float v = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
        if (accumulate)
            v += load_as(dbias, column, dtype);
        store_as(dbias, column, dtype, v);
    }
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
    int64_t strips = (int64_t(sm_count) * 6 + across - 1) / across;
    const int64_t most = (rows + 31) / 32;  // four rows a thread at least
    strips = strips < most ? strips : most;
    strips = strips < 1024 ? strips : 1024;
    return int(strips > 1 ? strips : 1);
}

int launch_linear_slope(const LinearSlope& a, void* stream)
{
    const dim3 grid(unsigned((a.columns + kSlopeColumns - 1) / kSlopeColumns), unsigned(a.strips));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const auto launch = [&](void (*kernel)(LinearSlope)) {
        return launch_early(kernel, grid, kSlopeThreads, 0, st, a);
    };
    switch (a.act) {
    case LINEAR_RELU: return launch(k_linear_slope<LINEAR_RELU>);
    case LINEAR_GELU: return launch(k_linear_slope<LINEAR_GELU>);
    case LINEAR_GELU_TANH: return launch(k_linear_slope<LINEAR_GELU_TANH>);
    case LINEAR_SILU: return launch(k_linear_slope<LINEAR_SILU>);
    default: return launch(k_linear_slope<LINEAR_NONE>);
    }
}

int launch_linear_bias_grad(const float* partials, int32_t strips, int64_t columns, void* dbias,
                            int32_t dtype, bool accumulate, void* stream)
{
    return launch_early(k_linear_bias_grad, dim3(unsigned((columns + 63) / 64)), kBiasThreads, 0,
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
