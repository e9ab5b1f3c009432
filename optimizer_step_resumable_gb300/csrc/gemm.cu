// gemm.cu -- tensor maps of the tiled product's operands.
#include "gemm.h"

#include <atomic>

#include <cuda_runtime.h>

namespace osr {

namespace {

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// The driver's function has one address, whatever the device.
std::atomic<EncodeTiled> encode_tiled{nullptr};

}  // namespace

int gemm_init()
{
    if (encode_tiled.load())
        return cudaSuccess;
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                           cudaEnableDefault, &found);
    if (e != cudaSuccess)
        return int(e);
    if (found != cudaDriverEntryPointSuccess || !f)
        return int(cudaErrorNotSupported);
    encode_tiled.store(reinterpret_cast<EncodeTiled>(f));
    return cudaSuccess;
}

int gemm_map(const GemmOperand& o, int rows, bool bf16, CUtensorMap* map)
{
    const EncodeTiled encode = encode_tiled.load();
    if (!encode)
        return int(cudaErrorNotSupported);
    const int64_t wide = o.across ? o.outer : o.inner, high = o.across ? o.inner : o.outer;
    const cuuint64_t extent[2] = {cuuint64_t(wide), cuuint64_t(high)};
    // a single row may be given any distance
    const int64_t apart = high > 1 ? o.stride : (wide + 7) / 8 * 8;
    const cuuint64_t stride[1] = {cuuint64_t(apart) * 2};
    // 64 elements are the 128 bytes of a swizzled row; across, further ones are
    // copies of their own
    const cuuint32_t box[2] = {64, cuuint32_t(o.across ? 64 : rows)};
    const cuuint32_t each[2] = {1, 1};
    const CUresult r = encode(
        map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
        const_cast<void*>(o.p), extent, stride, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? int(cudaSuccess) : int(cudaErrorInvalidValue);
}

}  // namespace osr
