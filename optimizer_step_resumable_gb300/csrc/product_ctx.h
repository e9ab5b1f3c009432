// product_ctx.h -- what the contexts of operators made of tiled products
// share: their device, the word in which a kernel says that a wait of its ran
// out, and the division of a call's workspace.
#pragma once

#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "api_util.h"
#include "arrays.h"
#include "gemm.h"
#include "linear.h"

namespace osr {

struct ProductContext {
    int device = -1;
    int sm_count = 0;
    int32_t* h_gave_up = nullptr;  // pinned, mapped
    int32_t* gave_up = nullptr;    // its device address
};

inline int product_create(ProductContext* c)
{
    cudaError_t e = cudaGetDevice(&c->device);
    if (e != cudaSuccess) {
        c->device = -1;
        return cuda_fail(e, "cudaGetDevice");
    }
    CUDA_TRY(cudaDeviceGetAttribute(&c->sm_count, cudaDevAttrMultiProcessorCount, c->device));
    e = cudaError_t(gemm_init());
    if (e != cudaSuccess)
        return cuda_fail(e, "cuTensorMapEncodeTiled");
    CUDA_TRY(cudaHostAlloc(reinterpret_cast<void**>(&c->h_gave_up), sizeof(int32_t),
                           cudaHostAllocMapped | cudaHostAllocPortable));
    *c->h_gave_up = 0;
    CUDA_TRY(cudaHostGetDevicePointer(reinterpret_cast<void**>(&c->gave_up), c->h_gave_up, 0));
    return ADAMW_OK;
}

// cudaFreeHost waits for the device's work.
inline void product_free(ProductContext* c)
{
    if (c->device >= 0 && c->h_gave_up) {
        DeviceScope scope(c->device);
        cudaFreeHost(c->h_gave_up);
    }
}

inline int product_state(ProductContext* c)
{
    volatile int32_t* const word = c->h_gave_up;
    if (!*word)
        return ADAMW_OK;
    *word = 0;
    return fail(ADAMW_ESTATE,
                "a kernel of an earlier call gave up waiting: its outputs are not valid");
}

// The plans of the last few different calls, which take as long to make as some
// launches: a training step calls forward and backward in turn, with one context
// (8192 x 768 to 768: with the last call's alone, the two in turn took 3.4 us more on
// the host than each of them repeated; so, none).
template <typename Needs, typename Plans>
class RecentPlans {
public:
    template <typename Make>
    const Plans& of(int64_t rows, const Needs& needs, const Make& make)
    {
        for (const Entry& e : entries_)
            if (e.rows == rows && std::memcmp(&e.needs, &needs, sizeof needs) == 0)
                return e.plans;
        Entry& e = entries_[next_];
        next_ = (next_ + 1) % kEntries;
        e.plans = make();
        e.rows = rows;
        e.needs = needs;
        return e.plans;
    }

private:
    static constexpr int kEntries = 4;
    struct Entry {
        int64_t rows = -1;
        Needs needs{};  // without gaps: compared byte by byte
        Plans plans;
    };
    Entry entries_[kEntries];
    int next_ = 0;
};

// Parts of a call's workspace, each on a 256-byte boundary.
class Workspace {
public:
    explicit Workspace(void* memory) : memory_(static_cast<char*>(memory)) {}
    void* take(int64_t bytes)
    {
        char* const p = memory_ ? memory_ + used_ : nullptr;
        used_ += (bytes + 255) / 256 * 256;
        return p;
    }
    int64_t bytes() const { return used_; }

private:
    char* memory_;
    int64_t used_ = 0;
};

template <int kOut, int kIn>
int check_workspace(void* memory, int64_t bytes, int64_t needed, const Pieces (&out)[kOut],
                    const Pieces (&in)[kIn])
{
    if (needed == 0)
        return ADAMW_OK;
    if (!memory)
        return fail(ADAMW_EINVAL, "d_workspace is NULL: the call needs %lld bytes",
                    (long long)needed);
    if (reinterpret_cast<uintptr_t>(memory) % 256)
        return fail(ADAMW_EINVAL, "d_workspace is not on a 256-byte boundary");
    if (bytes < needed)
        return fail(ADAMW_EINVAL, "workspace of %lld bytes: the call needs %lld", (long long)bytes,
                    (long long)needed);
    const Pieces all[] = {vector_of(memory, needed, 1, "d_workspace")};
    const int rc = check_apart(all, in);
    return rc == ADAMW_OK ? check_apart(all, out) : rc;
}

// A row's elements in whole 16-byte vectors.
inline int64_t whole(int64_t elements) { return (elements + 7) / 8 * 8; }

// Whether rows start on 32-byte boundaries.
inline bool on_vectors(const void* p, int64_t stride, int64_t rows, size_t size)
{
    return reinterpret_cast<uintptr_t>(p) % 32 == 0 &&
           (rows <= 1 || stride * int64_t(size) % 32 == 0);
}

// Makes p, rows of `columns` elements `stride` apart, one that the tiled copies
// can read: a copy of it in `copy`, unless that is NULL.  The copy is still to
// be made.
inline LinearCopy copy_of(const void** p, int64_t* stride, int64_t rows, int64_t columns,
                          void* copy)
{
    const LinearCopy c{*p, *stride, copy, whole(columns), rows, columns};
    if (copy) {
        *p = copy;
        *stride = whole(columns);
    }
    return c;
}
inline int copy_readable(const LinearCopy& a, const LinearCopy& b, void* stream)
{
    return a.to || b.to ? launch_linear_copies(a, b, stream) : int(cudaSuccess);
}

}  // namespace osr
