// fake_driver.cpp -- the one function of the driver that the library asks the
// runtime for, the encoder of tensor maps, in a form that notes what it is given
// and refuses what the real one refuses.
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime_api.h>

namespace {

int maps = 0, refused = 0;

CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t rank, void* address,
                const cuuint64_t* extent, const cuuint64_t* stride, const cuuint32_t* box,
                const cuuint32_t* each, CUtensorMapInterleave, CUtensorMapSwizzle,
                CUtensorMapL2promotion, CUtensorMapFloatOOBfill)
{
    ++maps;
    const bool good = rank == 2 && address && reinterpret_cast<uintptr_t>(address) % 16 == 0 &&
                      extent[0] >= 1 && extent[0] <= (uint64_t(1) << 32) && extent[1] >= 1 &&
                      extent[1] <= (uint64_t(1) << 32) && stride[0] % 16 == 0 &&
                      stride[0] < (uint64_t(1) << 40) && box[0] == 64 && box[1] >= 1 &&
                      box[1] <= 256 && each[0] == 1 && each[1] == 1;
    if (!good)
        ++refused;
    return good ? CUDA_SUCCESS : CUDA_ERROR_INVALID_VALUE;
}

}  // namespace

extern "C" {

int fake_maps(void) { return maps; }
int fake_maps_refused(void) { return refused; }

cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned int, unsigned long long,
                                             cudaDriverEntryPointQueryResult* found)
{
    *f = reinterpret_cast<void*>(&encode);
    *found = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}

}  // extern "C"
