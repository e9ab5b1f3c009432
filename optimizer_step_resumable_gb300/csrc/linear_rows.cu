// linear_rows.cu -- the linear layer's passes over rows: the gradient through
// the activation with the bias's gradient, and copies of rows that the tiled
// copies cannot read.  All are bound by memory: each value is read once.
#include "early_dev.cuh"
#include "linear_dev.cuh"

namespace osr {
namespace {

using namespace detail;

// A block has 256 neighbouring columns of a strip of the rows, a warp every
// eighth row, a thread eight neighbouring columns.  kAtOnce rows of a thread
// are on their way at a time.  The eight warps' sums of a column meet in shared
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
// A warp's 256 elements of a row from `p` on, eight neighbours a lane, of which
// there are `count` in all (the rest 0).  The row may start anywhere: the 16-byte
// pieces of memory that lie within it come as they are, those at its ends
// element by element, and a lane puts its eight together from two of them.
struct RowPiece {
    uint4 here, last;  // last: the one behind the warp's, in lane 31
};
__device__ __forceinline__ uint4 piece_of(const uint16_t* p, int32_t from, int32_t count)
{
    if (from >= 0 && from + 8 <= count)
        return __ldcs(reinterpret_cast<const uint4*>(p + from));
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = from + i >= 0 && from + i < count ? p[from + i] : 0u;
    return make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16),
                      w[6] | (w[7] << 16));
}
// Elements from the 16-byte boundary before p to p.
__device__ __forceinline__ int32_t cut_of(const uint16_t* p)
{
    return int32_t(reinterpret_cast<uintptr_t>(p) / 2 % 8);
}
__device__ __forceinline__ RowPiece load_piece(const uint16_t* p, int32_t count)
{
    const int lane = threadIdx.x % 32;
    const int32_t cut = cut_of(p);
    RowPiece r;
    r.here = piece_of(p, 8 * lane - cut, count);
    r.last = make_uint4(0, 0, 0, 0);
    if (lane == 31 && cut)
        r.last = piece_of(p, 256 - cut, count);
    return r;
}
// Of rows that start on 16-byte boundaries.
template <typename Piece>
__device__ __forceinline__ Piece load_as_piece(const uint16_t* p, int32_t count)
{
    if constexpr (std::is_same_v<Piece, RowPiece>)
        return load_piece(p, count);
    else
        return piece_of(p, 8 * (threadIdx.x % 32), count);
}
__device__ __forceinline__ uint4 join_piece(uint4 r, const uint16_t*) { return r; }
// For a whole warp, with the p that the piece was loaded from.
__device__ __forceinline__ uint4 join_piece(const RowPiece& r, const uint16_t* p)
{
    const int32_t cut = cut_of(p);
    if (cut == 0)
        return r.here;
    const bool end = threadIdx.x % 32 == 31;
    uint32_t w[8] = {r.here.x, r.here.y, r.here.z, r.here.w};
    const uint32_t last[4] = {r.last.x, r.last.y, r.last.z, r.last.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, w[i], 1);
        w[4 + i] = end ? last[i] : next;
    }
    // whole words, then half of one
    if (cut & 4)
#pragma unroll
        for (int i = 0; i < 6; ++i)
            w[i] = w[i + 2];
    if (cut & 2)
#pragma unroll
        for (int i = 0; i < 5; ++i)
            w[i] = w[i + 1];
    if (cut & 1)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// kRagged: rows of dy or z do not start on 16-byte boundaries.
template <int kAct, bool kRagged>
__global__ void __launch_bounds__(kSlopeThreads, 2) k_linear_slope(const LinearSlope a)
{
    __shared__ float sums[8][kSlopeColumns + 8];
    wait_before();
    go_ahead();
    constexpr int kAtOnce = kRagged ? 2 : 4;
    const int lane = threadIdx.x % 32, group = threadIdx.x / 32;
    const int64_t base = int64_t(blockIdx.x) * kSlopeColumns;
    const int32_t count = int32_t(a.columns - base < kSlopeColumns ? a.columns - base
                                                                   : kSlopeColumns);
    const int64_t first = a.rows * blockIdx.y / a.strips;
    const int64_t last = a.rows * (blockIdx.y + 1) / a.strips;
    const uint16_t* dy = static_cast<const uint16_t*>(a.dy) + (first + group) * a.dy_stride + base;
    const uint16_t* z = static_cast<const uint16_t*>(a.z) + (first + group) * a.z_stride + base;
    uint16_t* dz =
        static_cast<uint16_t*>(a.dz) + (first + group) * a.stride + base + 8 * lane;
    float total[8] = {};
    for (int64_t r = first + group; r < last; r += 8 * kAtOnce) {
        using Piece = std::conditional_t<kRagged, RowPiece, uint4>;
        Piece g[kAtOnce], x[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (r + 8 * k < last) {
                g[k] = load_as_piece<Piece>(dy + 8 * k * a.dy_stride, count);
                if constexpr (kAct != LINEAR_NONE)
                    x[k] = load_as_piece<Piece>(z + 8 * k * a.z_stride, count);
            }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (r + 8 * k < last) {
                float f[8];
                widen8(join_piece(g[k], dy + 8 * k * a.dy_stride), a.bf16, f);
                if constexpr (kAct != LINEAR_NONE) {
                    float s[8];
                    widen8(join_piece(x[k], z + 8 * k * a.z_stride), a.bf16, s);
                    times_slopes<kAct>(f, s);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    total[i] += f[i];
                // rows of whole vectors: the stride is a multiple of eight
                if (a.dz && 8 * lane < count)
                    *reinterpret_cast<uint4*>(dz + 8 * k * a.stride) =
                        make_uint4(narrow32(f[0], f[1], a.bf16), narrow32(f[2], f[3], a.bf16),
                                   narrow32(f[4], f[5], a.bf16), narrow32(f[6], f[7], a.bf16));
            }
        dy += 8 * kAtOnce * a.dy_stride;
        z += 8 * kAtOnce * a.z_stride;
        dz += 8 * kAtOnce * a.stride;
    }
    if (!a.partials)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sums[group][8 * lane + i] = total[i];
    __syncthreads();
    if (int32_t(threadIdx.x) < count) {
        float s = 0.0f;
#pragma unroll
        for (int g = 0; g < 8; ++g)
            s += sums[g][threadIdx.x];
        a.partials[blockIdx.y * a.columns + base + threadIdx.x] = s;
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

// A warp has 256 columns of every so many rows, four of them on their way.
constexpr int kCopyThreads = 256;
__global__ void __launch_bounds__(kCopyThreads)
    k_copy_rows(const uint16_t* from, int64_t from_stride, uint16_t* to, int64_t to_stride,
                int64_t rows, int64_t columns)
{
    wait_before();
    go_ahead();
    constexpr int kAtOnce = 4;
    const int lane = threadIdx.x % 32;
    const int64_t base = int64_t(blockIdx.x) * 256;
    const int32_t count = int32_t(columns - base < 256 ? columns - base : 256);
    const int64_t step = int64_t(gridDim.y) * (kCopyThreads / 32);
    from += base;
    to += base + 8 * lane;
    for (int64_t r = int64_t(blockIdx.y) * (kCopyThreads / 32) + threadIdx.x / 32; r < rows;
         r += kAtOnce * step) {
        RowPiece w[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (r + k * step < rows)
                w[k] = load_piece(from + (r + k * step) * from_stride, count);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (r + k * step < rows) {
                const uint4 v = join_piece(w[k], from + (r + k * step) * from_stride);
                if (8 * lane < count)
                    *reinterpret_cast<uint4*>(to + (r + k * step) * to_stride) = v;
            }
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
    const bool ragged =
        !gemm_readable(a.dy, a.rows > 1 ? a.dy_stride : 0) ||
        (a.act != LINEAR_NONE && !gemm_readable(a.z, a.rows > 1 ? a.z_stride : 0));
    const auto launch = [&](void (*even)(LinearSlope), void (*uneven)(LinearSlope)) {
        return launch_early(ragged ? uneven : even, grid, kSlopeThreads, 0,
                            static_cast<cudaStream_t>(stream), a);
    };
    switch (a.act) {
    case LINEAR_RELU:
        return launch(k_linear_slope<LINEAR_RELU, false>, k_linear_slope<LINEAR_RELU, true>);
    case LINEAR_GELU:
        return launch(k_linear_slope<LINEAR_GELU, false>, k_linear_slope<LINEAR_GELU, true>);
    case LINEAR_GELU_TANH:
        return launch(k_linear_slope<LINEAR_GELU_TANH, false>,
                      k_linear_slope<LINEAR_GELU_TANH, true>);
    case LINEAR_SILU:
        return launch(k_linear_slope<LINEAR_SILU, false>, k_linear_slope<LINEAR_SILU, true>);
    default: return launch(k_linear_slope<LINEAR_NONE, false>, k_linear_slope<LINEAR_NONE, true>);
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
    const int64_t across = (columns + 255) / 256;
    int64_t blocks = (rows + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    const int64_t most = across < 2048 ? 2048 / across : 1;
    blocks = blocks < most ? blocks : most;
    return launch_early(k_copy_rows, dim3(unsigned(across), unsigned(blocks)), kCopyThreads, 0,
                        static_cast<cudaStream_t>(stream), static_cast<const uint16_t*>(from),
                        from_stride, static_cast<uint16_t*>(to), to_stride, rows, columns);
}

}  // namespace osr
