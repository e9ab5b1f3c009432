// linear_gemm.cuh -- the epilogue of the linear layer's products, a translation
// unit for each type of the output.
#pragma once

#include "gemm.cuh"
#include "linear_dev.cuh"

namespace osr {

struct StoreParams {
    LinearOut o;
    int64_t rows, columns;
    int64_t split_stride;  // elements of out from one split's sums to the next's
};

// One product, ready for its tiles; its sums go where p says.
struct StoreProduct {
    GemmOperand a, b;
    GemmShape s;  // splits, chains
    StoreParams p;
    GemmSide side;  // of the first of two
};
// Tiles of 256 x bn (128, 192 or 256), the product's rows along the long side,
// for an output of the type; `plain`: neither bias nor activation nor z, which
// float32 outputs never have.
int linear_store_f32(int bn, const StoreProduct& p, bool bf16, int sm_count, void* stream);
int linear_store_bf16(int bn, const StoreProduct& p, bool plain, bool bf16, int sm_count,
                      void* stream);
int linear_store_f16(int bn, const StoreProduct& p, bool plain, bool bf16, int sm_count,
                     void* stream);
// Two plain products in one launch, in tiles of 256 x 256; the types of their
// outputs, float32 or bf16's 16-bit type.
int linear_store_two_f32(const StoreProduct& p, const StoreProduct& q, bool bf16,
                         const GemmDeal& deal, void* stream);
int linear_store_two_bf16(const StoreProduct& p, const StoreProduct& q, const GemmDeal& deal,
                          void* stream);
int linear_store_two_f16(const StoreProduct& p, const StoreProduct& q, const GemmDeal& deal,
                         void* stream);

namespace detail {

template <int kType>
constexpr int kSize = kType == ADAMW_DTYPE_F32 ? 4 : 2;
template <int kType>
__device__ __forceinline__ float get(const char* p)
{
    return load_as(p, 0, kType);
}

// The tile's rows are the product's: a thread has a row's neighbouring
// columns, 32 at a time.  Rows on 32-byte boundaries go out from each thread,
// whole sectors at a time, and what is added to them comes in the same way,
// two chunks ahead (one, if it is float32).  Rows of float32 go out four at a time
// instead, 128 bytes of each, through shared memory: a later chain's sums are
// added to them in L2.  Rows on other boundaries go through shared memory, so
// that a warp's lanes have neighbouring columns of one row, eight rows at a time.
// kPlain: neither bias nor activation nor z.
template <int kOut, bool kPlain>
struct StoreEpilogue {
    using Params = StoreParams;
    static constexpr int kUnroll = 4;
    static constexpr bool kF32 = kOut == ADAMW_DTYPE_F32, kBf16 = kOut == ADAMW_DTYPE_BF16;

    int32_t row, end_column;  // of the columns that are this thread's
    float alpha;
    bool vectors, again, add, add_f32, bias;
    char* out;        // the row
    const char* from;  // what is added to it
    float lane_bias[4];  // of the chunks, for the lane's column
    uint32_t ahead[32];

    __device__ StoreEpilogue(const Params& p, const GemmShape&, int32_t r, int32_t column,
                             int32_t count, const GemmItem& it, int32_t, float* stage)
        : row(r), end_column(column + count < p.columns ? column + count : int32_t(p.columns)),
          alpha(p.o.alpha), vectors(p.o.vectors), bias(!kPlain && p.o.bias)
    {
        const LinearOut& o = p.o;
        if (o.alpha_factor)
            alpha *= *o.alpha_factor;
        out = static_cast<char*>(o.out) +
              (it.split * p.split_stride + int64_t(r) * o.stride) * kSize<kOut>;
        // a later chain adds to what the one before it left there
        again = kF32 && it.chain > 0;
        add = again || o.residual;
        add_f32 = again || o.residual_dtype == ADAMW_DTYPE_F32;
        from = again ? out
                     : static_cast<const char*>(o.residual) +
                           int64_t(r) * o.residual_stride * (add_f32 ? 4 : 2);
        if (!kPlain && bias) {
            const int lane = threadIdx.x % 32;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                lane_bias[c] = column + 32 * c + lane < end_column
                                   ? load_as(o.bias, column + 32 * c + lane, o.bias_dtype)
                                   : 0.0f;
            if (vectors) {  // for all lanes to read
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    stage[32 * c + lane] = lane_bias[c];
                __syncwarp();
            }
        }
        if (kF32) {
            if (add && !again && vectors)
                fetch_strip(p, column);
        } else if (add && vectors) {
            fetch(p, column, 0);
            if (!add_f32)
                fetch(p, column + 32, 1);
        }
    }
    // What is added to the 32 columns from `column`; `slot`: of two, for the
    // 16-bit types.
    __device__ __forceinline__ void fetch(const Params& p, int32_t column, int slot)
    {
        if (row >= p.rows || column + 32 > end_column)
            return;
        if (add_f32) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                load32(from + (int64_t(column) + 8 * i) * 4,
                       *reinterpret_cast<uint32_t(*)[8]>(ahead + 8 * i));
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                load32(from + (int64_t(column) + 16 * i) * 2,
                       *reinterpret_cast<uint32_t(*)[8]>(ahead + 16 * slot + 8 * i));
        }
    }
    // float32, in the strip's order: a lane has four neighbouring columns of every
    // fourth row, from row lane / 8 of the warp's.
    __device__ __forceinline__ void fetch_strip(const Params& p, int32_t column)
    {
        if (column + 32 > end_column)
            return;
        const int32_t lane = threadIdx.x % 32, r = row - lane + lane / 8;
        const int64_t step = p.o.residual_stride * 4;
        const char* at = from + (lane / 8 - lane) * step + (int64_t(column) + 4 * (lane % 8)) * 4;
#pragma unroll
        for (int i = 0; i < 32; i += 4)
            if (r + i < p.rows) {
                const uint4 w = *reinterpret_cast<const uint4*>(at + i * step);
                ahead[i] = w.x, ahead[i + 1] = w.y, ahead[i + 2] = w.z, ahead[i + 3] = w.w;
            }
    }
    __device__ __forceinline__ void store_strip(const Params& p, int32_t column,
                                                const float (&v)[32], uint4* strip)
    {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            strip_put(strip, i, make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                           __float_as_uint(v[4 * i + 2]),
                                           __float_as_uint(v[4 * i + 3])));
        __syncwarp();
        const int32_t lane = threadIdx.x % 32, piece = lane % 8, first = row - lane;
        const int64_t step = p.o.stride * 4;
        char* to = out - lane * step + (int64_t(column) + 4 * piece) * 4;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const int32_t r = i + lane / 8;
            const uint4 w = strip[8 * r + (piece ^ (r & 7))];
            float4 f = make_float4(__uint_as_float(w.x), __uint_as_float(w.y),
                                   __uint_as_float(w.z), __uint_as_float(w.w));
            if (first + r >= p.rows)
                continue;
            if (again) {
                add_to(to + r * step, f);
                continue;
            }
            if (add) {
                f.x += __uint_as_float(ahead[i]), f.y += __uint_as_float(ahead[i + 1]);
                f.z += __uint_as_float(ahead[i + 2]), f.w += __uint_as_float(ahead[i + 3]);
            }
            *reinterpret_cast<float4*>(to + r * step) = f;
        }
        if (add && !again)
            fetch_strip(p, column + 32);
    }
    // Adds where the values lie: nothing comes back.  A place belongs to one
    // thread in every chain of its tile, so the order is the chains'.
    __device__ static __forceinline__ void add_to(char* p, float4 f)
    {
        asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(f.x),
                     "f"(f.y), "f"(f.z), "f"(f.w)
                     : "memory");
    }
    __device__ static __forceinline__ void store(char* to, const float (&v)[32])
    {
        uint32_t w[8];
        if constexpr (kF32) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = __float_as_uint(v[i + j]);
                store32(to + i * 4, w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; i += 16) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = narrow32(v[i + 2 * j], v[i + 2 * j + 1], kBf16);
                store32(to + i * 2, w);
            }
        }
    }
    template <int C>
    __device__ __forceinline__ void chunk(const Params& p, const GemmShape&, int32_t column, int c,
                                          float (&v)[C], float* stage)
    {
        static_assert(C == 32, "");
        const LinearOut& o = p.o;
        if (column >= p.columns)
            return;
        if (alpha != 1.0f)
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] *= alpha;
        if (kF32 && vectors && column + 32 <= p.columns) {
            store_strip(p, column, v, reinterpret_cast<uint4*>(stage));
            return;
        }
        if (vectors && column + 32 <= p.columns) {
            if (!kPlain && bias)
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 b = *reinterpret_cast<const float4*>(stage + 32 * c + i);
                    v[i] += b.x, v[i + 1] += b.y, v[i + 2] += b.z, v[i + 3] += b.w;
                }
            if (!kPlain && o.z && row < p.rows)
                store(static_cast<char*>(o.z) + (int64_t(row) * o.z_stride + column) * kSize<kOut>,
                      v);
            if (!kPlain && o.act != LINEAR_NONE)
                with_activation(o.act, [&](auto act) { activate_all<decltype(act)::value>(v); });
            if (add) {
                if (add_f32) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[i] += __uint_as_float(ahead[i]);
                    fetch(p, column + 32, 0);
                } else {
                    // float32 products add 16-bit values nowhere
                    if constexpr (!kF32) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint32_t w = ahead[16 * (c & 1) + i];
                            v[2 * i] += widen16(w & 0xFFFFu, kBf16);
                            v[2 * i + 1] += widen16(w >> 16, kBf16);
                        }
                    }
                    fetch(p, column + 64, c & 1);
                }
            }
            if (row < p.rows)
                store(out + int64_t(column) * kSize<kOut>, v);
            return;
        }
        const int lane = threadIdx.x % 32;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i)
            stage[lane * 33 + i] = v[i];
        __syncwarp();
        // the warp's rows, from its first lane's
        const int32_t left = p.rows - (row - lane) < 32 ? int32_t(p.rows - (row - lane)) : 32;
        const int32_t mine = column + lane;
        if (mine < p.columns) {
            const int64_t out_step = o.stride * kSize<kOut>, z_step = o.z_stride * kSize<kOut>;
            const int64_t add_step = (from == out ? o.stride : o.residual_stride) *
                                     (add_f32 ? 4 : 2);
            char* to = out - lane * out_step + int64_t(mine) * kSize<kOut>;
            const char* more = from - lane * add_step + int64_t(mine) * (add_f32 ? 4 : 2);
            char* z = static_cast<char*>(o.z) +
                      (int64_t(row - lane) * o.z_stride + mine) * kSize<kOut>;
            const float b = !kPlain && bias ? lane_bias[c] : 0.0f;
            for (int r = 0; r < left; r += 8) {
                float f[8], a[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    f[i] = stage[(r + i) * 33 + lane] + b;
                    a[i] = 0.0f;
                }
                if (add) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (r + i < left)
                            a[i] = add_f32 ? get<ADAMW_DTYPE_F32>(more + i * add_step)
                                           : get<kF32 ? ADAMW_DTYPE_BF16 : kOut>(more +
                                                                                 i * add_step);
                    more += 8 * add_step;
                }
                if (!kPlain && o.z) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (r + i < left)
                            store_as(z + i * z_step, 0, kOut, f[i]);
                    z += 8 * z_step;
                }
                if (!kPlain && o.act != LINEAR_NONE)
                    with_activation(o.act,
                                    [&](auto act) { activate_all<decltype(act)::value>(f); });
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (r + i < left)
                        store_as(to + i * out_step, 0, kOut, f[i] + a[i]);
                to += 8 * out_step;
            }
        }
        __syncwarp();
    }
    __device__ void end(const Params&, const GemmShape&) {}
};

template <int kOut, int kOut2>
inline int store_two(const StoreProduct& p, const StoreProduct& q, bool bf16,
                     const GemmDeal& deal, void* stream)
{
    using E = StoreEpilogue<kOut, true>;
    using E2 = StoreEpilogue<kOut2, true>;
    GemmPart<E> one;
    GemmPart<E2> two;
    int e = gemm_part<256, E>(p.a, p.b, p.s, bf16, p.p, &one);
    if (e == cudaSuccess)
        e = gemm_part<256, E2>(q.a, q.b, q.s, bf16, q.p, &two);
    return e == cudaSuccess
               ? gemm_launch<256, E, E2>(one, two, deal, p.side, static_cast<cudaStream_t>(stream))
               : e;
}
template <int kOut, bool kPlain>
inline int store_one(int bn, const StoreProduct& p, bool bf16, int sm_count, void* stream)
{
    using E = StoreEpilogue<kOut, kPlain>;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (bn) {
    case 128: return gemm_run<128, E>(p.a, p.b, p.s, bf16, p.p, p.side, sm_count, st);
    case 192: return gemm_run<192, E>(p.a, p.b, p.s, bf16, p.p, p.side, sm_count, st);
    default: return gemm_run<256, E>(p.a, p.b, p.s, bf16, p.p, p.side, sm_count, st);
    }
}

}  // namespace detail
}  // namespace osr
