// fake_cudart.cpp -- a CUDA runtime of two devices that run nothing, for tests
// of the library's host code: it keeps, per device, how much dynamic shared
// memory each kernel was allowed, refuses launches beyond it, notes every
// launch's grid, and fails calls when told to.
#include <cstdlib>
#include <cstring>
#include <map>
#include <utility>

#include <cuda_runtime_api.h>

namespace {

constexpr int kDevices = 2;
constexpr int kSms[kDevices] = {152, 100}, kBlocks[kDevices] = {3, 2};
constexpr size_t kDefaultSmem = 48 * 1024;

int current = 0;
int fail_attribute = 0, fail_occupancy = 0;  // calls that still fail
std::map<std::pair<int, const void*>, size_t> allowed;
int launches = 0, last_device = -1;
unsigned last_blocks = 0;

size_t allowance(const void* f)
{
    const auto it = allowed.find({current, f});
    return it == allowed.end() ? kDefaultSmem : it->second;
}

}  // namespace

extern "C" {

// ---- the test's own calls ----
void fake_fail(int attribute_calls, int occupancy_calls)
{
    fail_attribute = attribute_calls;
    fail_occupancy = occupancy_calls;
}
int fake_launches(void) { return launches; }
int fake_last_device(void) { return last_device; }
unsigned fake_last_blocks(void) { return last_blocks; }
int fake_sms(int device) { return kSms[device]; }
int fake_blocks(int device) { return kBlocks[device]; }

// ---- the runtime's ----
cudaError_t cudaGetDevice(int* device)
{
    *device = current;
    return cudaSuccess;
}
cudaError_t cudaSetDevice(int device)
{
    if (device < 0 || device >= kDevices)
        return cudaErrorInvalidDevice;
    current = device;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* value, cudaDeviceAttr, int device)
{
    *value = kSms[device];
    return cudaSuccess;
}
cudaError_t cudaMalloc(void** p, size_t bytes)
{
    *p = std::aligned_alloc(256, (bytes + 255) / 256 * 256);
    return cudaSuccess;
}
cudaError_t cudaFree(void* p)
{
    std::free(p);
    return cudaSuccess;
}
cudaError_t cudaHostAlloc(void** p, size_t bytes, unsigned) { return cudaMalloc(p, bytes); }
cudaError_t cudaFreeHost(void* p) { return cudaFree(p); }
cudaError_t cudaHostGetDevicePointer(void** d, void* h, unsigned)
{
    *d = h;
    return cudaSuccess;
}
cudaError_t cudaMemcpy(void* to, const void* from, size_t bytes, cudaMemcpyKind)
{
    std::memcpy(to, from, bytes);
    return cudaSuccess;
}
cudaError_t cudaMemset(void* p, int value, size_t bytes)
{
    std::memset(p, value, bytes);
    return cudaSuccess;
}
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s)
{
    *s = cudaStreamCaptureStatusNone;
    return cudaSuccess;
}
const char* cudaGetErrorName(cudaError_t) { return "name"; }
const char* cudaGetErrorString(cudaError_t) { return "text"; }
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int value)
{
    if (fail_attribute > 0) {
        --fail_attribute;
        return cudaErrorUnknown;
    }
    allowed[{current, f}] = size_t(value);
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void* f, int,
                                                                   size_t smem, unsigned)
{
    if (fail_occupancy > 0) {
        --fail_occupancy;
        return cudaErrorUnknown;
    }
    *n = smem <= allowance(f) ? kBlocks[current] : 0;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void* f, int threads,
                                                          size_t smem)
{
    return cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(n, f, threads, smem, 0);
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**)
{
    if (c->dynamicSmemBytes > allowance(f))
        return cudaErrorInvalidValue;
    ++launches;
    last_device = current;
    last_blocks = c->gridDim.x;
    return cudaSuccess;
}

}  // extern "C"
