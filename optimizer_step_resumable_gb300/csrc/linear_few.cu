// linear_few.cu -- the linear layer for a few rows, as when tokens are generated
// one at a time: what bounds it is reading the weight once.
//
// A tensor core tile of 256 rows would be empty but for one; here a thread
// multiplies what it has just read, in float32, and there is one launch, with no
// sums to join.  It pays for one or two rows, and for up to eight where the
// weight is small and launches are the time (linear_few_pays).  us on the GPU,
// bf16, weight stored (out, in), in place of tiles: 1 x 2048 x 8192 8.3 (10.5 in
// tiles; its 34 MB take 4.9), 2 x 4096 x 16384 30 (24), 1 x 768 x 768 1.9 (6.1), 8 x
// 768 x 768 3.9; but 8 x 2048 x 8192 40.  Stored (in, out): 1 x 768 x 768 3.2, but 1 x
// 2048 x 8192 12.6.
#include "early_dev.cuh"
#include "linear_dev.cuh"

namespace osr {
namespace {

using namespace detail;
using packed::fma2;

struct FewParams {
    LinearOut o;
    const uint16_t* x;
    int64_t x_stride;
    const uint16_t* weight;
    int64_t weight_stride;
    int64_t columns, inner;
    int32_t rows;
    bool bf16;
};

__device__ __forceinline__ void widen_pairs(uint4 q, bool bf16, float2 (&f)[4])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = make_float2(widen16(w[i] & 0xFFFFu, bf16), widen16(w[i] >> 16, bf16));
}
// Eight elements from place k of n; others 0.
__device__ __forceinline__ uint4 eight(const uint16_t* p, int64_t k, int64_t n)
{
    if (k + 8 <= n)
        return *reinterpret_cast<const uint4*>(p + k);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = k + i < n ? p[k + i] : 0u;
    return make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16),
                      w[6] | (w[7] << 16));
}

// Rows of the weight lie along the sum: a group of kShare warps has kOuts of
// them, its warps every kShare-th vector of 32 lanes.
constexpr int kAlongThreads = 128, kAlongWarps = kAlongThreads / 32;
template <int M, int kOuts, int kShare>
__global__ void __launch_bounds__(kAlongThreads) k_linear_few_along(const FewParams p)
{
    __shared__ float slots[kAlongWarps][M * kOuts];
    wait_before();
    go_ahead();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, part = warp % kShare;
    const int64_t first =
        (int64_t(blockIdx.x) * (kAlongWarps / kShare) + warp / kShare) * kOuts;
    float2 sum[M][kOuts] = {};
    if (first < p.columns)
#pragma unroll(M <= 2 ? 4 : 2)
        for (int64_t k = 8 * (lane + 32 * part); k < p.inner; k += 256 * kShare) {
            float2 w[kOuts][4];
#pragma unroll
            for (int o = 0; o < kOuts; ++o) {
                // the last outputs again, where there are no more
                const int64_t out = first + o < p.columns ? first + o : p.columns - 1;
                widen_pairs(eight(p.weight + out * p.weight_stride, k, p.inner), p.bf16, w[o]);
            }
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if (m >= p.rows)
                    break;
                float2 x[4];
                widen_pairs(eight(p.x + m * p.x_stride, k, p.inner), p.bf16, x);
#pragma unroll
                for (int o = 0; o < kOuts; ++o)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sum[m][o] = fma2(w[o][i], x[i], sum[m][o]);
            }
        }
    float mine = 0.0f;  // of row lane / kOuts, output lane % kOuts
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int o = 0; o < kOuts; ++o) {
            float s = sum[m][o].x + sum[m][o].y;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
            mine = lane == m * kOuts + o ? s : mine;
        }
    if constexpr (kShare > 1) {
        if (lane < M * kOuts)
            slots[warp][lane] = mine;
        __syncthreads();
        if (part > 0 || lane >= M * kOuts)
            return;
        mine = 0.0f;
#pragma unroll
        for (int i = 0; i < kShare; ++i)
            mine += slots[warp + i][lane];
    }
    const int64_t row = lane / kOuts, column = first + lane % kOuts;
    if (lane < M * kOuts && row < p.rows && column < p.columns) {
        const LinearOut o = with_factor(p.o);
        with_activation(o.act, [&](auto act) {
            float v[1] = {mine};
            finish_some<decltype(act)::value>(o, row, column, v);
        });
    }
}

// Rows of the weight lie across the sum: a block has 64 columns, a warp four
// rows of them at a time, eight columns a thread; the blocks of a cluster have
// a share of the rows each and join their sums through one another's shared
// memory.
constexpr int kAcrossThreads = 256, kAcrossWarps = kAcrossThreads / 32, kAcrossColumns = 64;
template <int M>
__global__ void __launch_bounds__(kAcrossThreads) k_linear_few_across(const FewParams p)
{
    __shared__ float sums[kAcrossWarps][M][kAcrossColumns];
    wait_before();
    go_ahead();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t base = int64_t(blockIdx.x) * kAcrossColumns, column = base + 8 * (lane % 8);
    const int64_t begin = p.inner * blockIdx.y / gridDim.y;
    const int64_t end = p.inner * (blockIdx.y + 1) / gridDim.y;
    float2 sum[M][4] = {};
    if (column < p.columns)
#pragma unroll(M <= 2 ? 8 : 4)
        for (int64_t k = begin + 4 * warp + lane / 8; k < end; k += 4 * kAcrossWarps) {
            float2 w[4];
            widen_pairs(eight(p.weight + k * p.weight_stride, column, p.columns), p.bf16, w);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if (m >= p.rows)
                    break;
                const float x = widen16(p.x[m * p.x_stride + k], p.bf16);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum[m][i] = fma2(w[i], packed::both(x), sum[m][i]);
            }
        }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 s = sum[m][i];
#pragma unroll
            for (int off = 8; off < 32; off *= 2) {
                s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, off);
                s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, off);
            }
            if (lane < 8)
                *reinterpret_cast<float2*>(&sums[warp][m][8 * lane + 2 * i]) = s;
        }
    __syncthreads();
    // the block's sum, in the first warp's place
    for (int i = threadIdx.x; i < M * kAcrossColumns; i += kAcrossThreads) {
        const int m = i / kAcrossColumns, c = i % kAcrossColumns;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kAcrossWarps; ++w)
            s += sums[w][m][c];
        sums[0][m][c] = s;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
    // each block finishes its part of the columns
    const LinearOut o = with_factor(p.o);
    const int each = kAcrossColumns / int(gridDim.y);
    for (int i = threadIdx.x; i < each * p.rows; i += kAcrossThreads) {
        const int m = i / each, c = int(blockIdx.y) * each + i % each;
        if (base + c >= p.columns)
            continue;
        const uint32_t here = uint32_t(__cvta_generic_to_shared(&sums[0][m][c]));
        float v[1] = {0.0f};
        for (uint32_t b = 0; b < gridDim.y; ++b) {
            uint32_t there;
            float s;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(b));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(s) : "r"(there) : "memory");
            v[0] += s;
        }
        with_activation(o.act, [&](auto act) {
            finish_some<decltype(act)::value>(o, m, base + c, v);
        });
    }
    // no block leaves while another reads its sums
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

template <int M, int kOuts>
int run_along(const FewParams& p, int sm_count, cudaStream_t stream)
{
    // several warps to an output where there are few outputs
    const int64_t groups = (p.columns + kOuts - 1) / kOuts;
    const bool share = groups < int64_t(sm_count) * 8 && p.inner > 512;
    const int64_t blocks = share ? groups : (groups + kAlongWarps - 1) / kAlongWarps;
    return launch_early(share ? k_linear_few_along<M, kOuts, kAlongWarps>
                              : k_linear_few_along<M, kOuts, 1>,
                        dim3(unsigned(blocks)), kAlongThreads, 0, stream, p);
}
template <int M>
int run_across(const FewParams& p, int sm_count, cudaStream_t stream)
{
    const int64_t parts = (p.columns + kAcrossColumns - 1) / kAcrossColumns;
    int cluster = 1;
    while (cluster < 8 && parts * cluster < 2 * int64_t(sm_count) && p.inner >= 64 * cluster)
        cluster *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(parts), unsigned(cluster));
    cfg.blockDim = dim3(kAcrossThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = unsigned(cluster);
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return int(cudaLaunchKernelEx(&cfg, k_linear_few_across<M>, p));
}

}  // namespace

bool linear_few_pays(const LinearSize& p)
{
    const bool small = p.columns * p.inner <= int64_t(1) << 21;
    if (p.a_across)
        return false;
    return p.b_across ? small && p.rows <= 4
                      : p.rows <= 1 || (p.rows <= 2 && p.columns * p.inner <= int64_t(1) << 25) ||
                            (small && p.rows <= 8);
}

int linear_few(const LinearProduct& m, int sm_count, void* stream)
{
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const FewParams p{m.to,
                      static_cast<const uint16_t*>(m.a.p),
                      m.a.stride,
                      static_cast<const uint16_t*>(m.b.p),
                      m.b.stride,
                      m.b.outer,
                      m.b.inner,
                      int32_t(m.a.outer),
                      m.bf16};
    if (m.b.across)
        return p.rows == 1   ? run_across<1>(p, sm_count, st)
               : p.rows == 2 ? run_across<2>(p, sm_count, st)
                             : run_across<4>(p, sm_count, st);
    return p.rows == 1   ? run_along<1, 2>(p, sm_count, st)
           : p.rows == 2 ? run_along<2, 2>(p, sm_count, st)
           : p.rows <= 4 ? run_along<4, 4>(p, sm_count, st)
                         : run_along<8, 4>(p, sm_count, st);
}

}  // namespace osr
