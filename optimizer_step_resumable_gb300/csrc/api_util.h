// api_util.h -- helpers shared by the files that define C ABI entry points.
#pragma once

#include <cuda_runtime.h>

#include "internal.h"

namespace osr {

inline int cuda_fail(cudaError_t e, const char* what)
{
    return fail(ADAMW_ECUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

#define CUDA_TRY(expr)                                      \
    do {                                                    \
        cudaError_t e_ = (expr);                            \
        if (e_ != cudaSuccess)                              \
            return osr::cuda_fail(e_, #expr);               \
    } while (0)

// Makes a device current for the scope of one call and restores the caller's
// device afterwards.
class DeviceScope {
public:
    explicit DeviceScope(int device)
    {
        if (cudaGetDevice(&prev_) != cudaSuccess)
            prev_ = -1;
        if (prev_ != device && cudaSetDevice(device) == cudaSuccess)
            switched_ = true;
    }
    ~DeviceScope()
    {
        if (switched_ && prev_ >= 0)
            cudaSetDevice(prev_);
    }
    DeviceScope(const DeviceScope&) = delete;
    DeviceScope& operator=(const DeviceScope&) = delete;

private:
    int prev_ = -1;
    bool switched_ = false;
};

}  // namespace osr
