// list_api.cu -- the C ABI entry points of the step over a list of tensors
// (adamw_list_* of include/adamw_ckpt.h): the table of tensors and of warps'
// units in device memory, the checks of the arrays, the two launches.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include <cuda_runtime.h>

#include "api_util.h"
#include "internal.h"
#include "list.h"

struct adamw_list {
    int device = -1;
    int sm_count = 0;
    std::vector<int64_t> numels;
    std::vector<uint8_t> state8, decay;
    std::vector<osr::ListTensor> tensors;
    int32_t n_units = 0, n_plain = 0;  // units, and those of 32-bit states
    double beta1 = 0.9, beta2 = 0.999, eps = 1e-8;

    // one allocation: [NormResult | counters x 4 | pad][partials][tensors][units]
    unsigned char* d_scratch = nullptr;
    osr::ListTensor* d_tensors = nullptr;
    osr::ListUnit* d_units = nullptr;
    osr::NormResult* h_res = nullptr;    // pinned, mapped
    osr::NormResult* h_res_dev = nullptr;
    cudaEvent_t ev_norm = nullptr;
    bool bound = false, launched = false;
    int32_t g_dtype = ADAMW_DTYPE_F32, w_lp_dtype = ADAMW_DTYPE_BF16;
    osr::ListBlocks most{};  // of the bound g_dtype's kernels

    static constexpr size_t kHead = 256;
    osr::NormResult* d_res() const { return reinterpret_cast<osr::NormResult*>(d_scratch); }
    uint32_t* d_counters() const { return reinterpret_cast<uint32_t*>(d_scratch + kHead / 2); }
    double* d_partials() const { return reinterpret_cast<double*>(d_scratch + kHead); }
};

namespace {

using osr::cuda_fail;
using osr::DeviceScope;
using osr::fail;

void free_list(adamw_list* l)
{
    if (!l)
        return;
    if (l->device >= 0) {
        DeviceScope scope(l->device);
        if (l->ev_norm && l->launched)
            cudaEventSynchronize(l->ev_norm);
        if (l->ev_norm) cudaEventDestroy(l->ev_norm);
        if (l->d_scratch) cudaFree(l->d_scratch);
        if (l->h_res) cudaFreeHost(l->h_res);
    }
    delete l;
}

int create_list(int32_t n_tensors, const int64_t* numels, const uint8_t* state8, adamw_list* l)
{
    std::vector<osr::ListUnit> units, eight;
    int64_t block0 = 0;
    for (int32_t k = 0; k < n_tensors; ++k) {
        if (numels[k] < 0 || numels[k] > INT32_MAX)
            return fail(ADAMW_EINVAL, "tensor %d has numel %lld, outside [0, 2^31-1]", k,
                        (long long)numels[k]);
        l->numels.push_back(numels[k]);
        l->state8.push_back(state8 && state8[k] ? 1 : 0);
        l->decay.push_back(1);
        osr::ListTensor t{};
        t.numel = int32_t(numels[k]);
        t.block0 = block0;
        l->tensors.push_back(t);
        block0 += (numels[k] + osr::kBlockElems - 1) / osr::kBlockElems;
        const int64_t n_units = (numels[k] + osr::kUnitElems - 1) / osr::kUnitElems;
        for (int64_t u = 0; u < n_units; ++u)
            (l->state8.back() ? eight : units).push_back(osr::ListUnit{k, int32_t(u)});
    }
    // the kernels count units in int32 and look a few grid strides ahead
    if (units.size() + eight.size() > size_t(1) << 30)
        return fail(ADAMW_EINVAL, "the list has more than 2^30 units of %d elements",
                    osr::kUnitElems);
    l->n_plain = int32_t(units.size());
    units.insert(units.end(), eight.begin(), eight.end());
    l->n_units = int32_t(units.size());

    cudaError_t e = cudaGetDevice(&l->device);
    if (e != cudaSuccess) {
        l->device = -1;
        return cuda_fail(e, "cudaGetDevice");
    }
    CUDA_TRY(cudaDeviceGetAttribute(&l->sm_count, cudaDevAttrMultiProcessorCount, l->device));
    static_assert(sizeof(osr::NormResult) <= adamw_list::kHead / 2, "scratch head layout");
    static_assert(alignof(osr::ListTensor) <= 16 && adamw_list::kHead % 16 == 0 &&
                      sizeof(double) * osr::kNormBlocksMax % 16 == 0,
                  "scratch layout");
    const size_t partials = sizeof(double) * osr::kNormBlocksMax;
    const size_t table = sizeof(osr::ListTensor) * size_t(n_tensors);
    CUDA_TRY(cudaMalloc(&l->d_scratch, adamw_list::kHead + partials + table +
                                           sizeof(osr::ListUnit) * units.size()));
    l->d_tensors =
        reinterpret_cast<osr::ListTensor*>(l->d_scratch + adamw_list::kHead + partials);
    l->d_units = reinterpret_cast<osr::ListUnit*>(l->d_tensors + n_tensors);
    // adamw_list_bind waits for these before the first step
    CUDA_TRY(cudaMemset(l->d_scratch, 0, adamw_list::kHead + partials));
    CUDA_TRY(cudaMemcpy(l->d_units, units.data(), sizeof(osr::ListUnit) * units.size(),
                        cudaMemcpyHostToDevice));
    CUDA_TRY(cudaHostAlloc(reinterpret_cast<void**>(&l->h_res), sizeof(osr::NormResult),
                           cudaHostAllocMapped));
    std::memset(l->h_res, 0, sizeof(osr::NormResult));
    CUDA_TRY(cudaHostGetDevicePointer(reinterpret_cast<void**>(&l->h_res_dev), l->h_res, 0));
    CUDA_TRY(cudaEventCreateWithFlags(&l->ev_norm, cudaEventDisableTiming));
    return ADAMW_OK;
}

// Copies the host's table to the device, once no step still reads the old
// one, and waits for it: a step may follow on any stream.
int upload(adamw_list* l)
{
    DeviceScope scope(l->device);
    CUDA_TRY(cudaDeviceSynchronize());
    CUDA_TRY(cudaMemcpy(l->d_tensors, l->tensors.data(),
                        sizeof(osr::ListTensor) * l->tensors.size(), cudaMemcpyHostToDevice));
    CUDA_TRY(cudaDeviceSynchronize());
    return ADAMW_OK;
}

struct Range {
    uintptr_t begin, end;
    int32_t tensor;
    const char* name;
};

// One array of tensor k: present, aligned to its elements; noted in `ranges`.
int check_array(const void* p, int64_t count, size_t size, int32_t k, const char* name,
                std::vector<Range>* ranges)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (!p)
        return fail(ADAMW_EINVAL, "%s[%d] is NULL", name, k);
    if (a % size)
        return fail(ADAMW_EINVAL, "%s[%d] is not %d-byte aligned", name, k, int(size));
    ranges->push_back(Range{a, a + size_t(count) * size, k, name});
    return ADAMW_OK;
}

int bind_list(adamw_list* l, float* const* d_w, void* const* d_g, int32_t g_dtype,
              void* const* d_m, void* const* d_v, float* const* d_m_scale,
              float* const* d_v_scale, void* const* d_w_lp, int32_t w_lp_dtype)
{
    const size_t gs = g_dtype == ADAMW_DTYPE_F32 ? 4 : 2;
    std::vector<osr::ListTensor> table(l->tensors);
    std::vector<Range> ranges;
    for (size_t i = 0; i < table.size(); ++i) {
        osr::ListTensor& t = table[i];
        const int32_t k = int32_t(i);
        const int64_t n = t.numel;
        t.flags = l->decay[i] ? osr::kListDecay : 0u;
        if (n == 0)
            continue;
        const int64_t blocks = (n + osr::kBlockElems - 1) / osr::kBlockElems;
        const size_t ss = l->state8[i] ? 1 : 4;
        int rc;
        if ((rc = check_array(d_w[i], n, 4, k, "d_w", &ranges)) ||
            (rc = check_array(d_g[i], n, gs, k, "d_g", &ranges)) ||
            (rc = check_array(d_m[i], n, ss, k, "d_m", &ranges)) ||
            (rc = check_array(d_v[i], n, ss, k, "d_v", &ranges)))
            return rc;
        t.w = d_w[i];
        t.g = d_g[i];
        t.m = d_m[i];
        t.v = d_v[i];
        t.m_scale = t.v_scale = nullptr;
        t.w_lp = nullptr;
        if (l->state8[i]) {
            if (!d_m_scale || !d_v_scale)
                return fail(ADAMW_EINVAL, "tensor %d has 8-bit states: it needs block scales", k);
            if ((rc = check_array(d_m_scale[i], blocks, 4, k, "d_m_scale", &ranges)) ||
                (rc = check_array(d_v_scale[i], blocks, 4, k, "d_v_scale", &ranges)))
                return rc;
            t.m_scale = d_m_scale[i];
            t.v_scale = d_v_scale[i];
        }
        if (d_w_lp) {
            if ((rc = check_array(d_w_lp[i], n, 2, k, "d_w_lp", &ranges)))
                return rc;
            t.w_lp = d_w_lp[i];
        }
        auto at = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; };
        if (at(t.w, 32) && at(t.g, 8 * gs) && at(t.m, 8 * ss) && at(t.v, 8 * ss) && at(t.w_lp, 16))
            t.flags |= osr::kListVec;
    }
    std::sort(ranges.begin(), ranges.end(),
              [](const Range& a, const Range& b) { return a.begin < b.begin; });
    for (size_t i = 1; i < ranges.size(); ++i)
        if (ranges[i].begin < ranges[i - 1].end)
            return fail(ADAMW_EINVAL, "%s[%d] overlaps %s[%d]", ranges[i].name, ranges[i].tensor,
                        ranges[i - 1].name, ranges[i - 1].tensor);
    osr::ListBlocks most;
    {
        DeviceScope scope(l->device);
        const int e = osr::list_step_blocks(g_dtype, l->sm_count, &most);
        if (e != cudaSuccess)
            return cuda_fail(cudaError_t(e), "the update's blocks per SM");
    }
    l->bound = false;
    l->most = most;
    l->tensors.swap(table);
    const int rc = upload(l);
    if (rc != ADAMW_OK)
        return rc;
    l->g_dtype = g_dtype;
    l->w_lp_dtype = w_lp_dtype;
    l->bound = true;
    return ADAMW_OK;
}

}  // namespace

extern "C" {

int adamw_list_create(int32_t n_tensors, const int64_t* numels, const uint8_t* state8,
                      adamw_list** out)
{
    osr::clear_error();
    if (!out)
        return fail(ADAMW_EINVAL, "out is NULL");
    *out = nullptr;
    if (n_tensors < 0 || (n_tensors > 0 && !numels))
        return fail(ADAMW_EINVAL, "n_tensors=%d, numels %s", n_tensors, numels ? "given" : "NULL");
    adamw_list* l = new (std::nothrow) adamw_list;
    if (!l)
        return fail(ADAMW_EINVAL, "out of host memory");
    int rc;
    try {
        rc = create_list(n_tensors, numels, state8, l);
    } catch (const std::bad_alloc&) {
        rc = fail(ADAMW_EINVAL, "out of host memory");
    }
    if (rc != ADAMW_OK) {
        free_list(l);
        return rc;
    }
    *out = l;
    return ADAMW_OK;
}

int adamw_list_destroy(adamw_list* list)
{
    osr::clear_error();
    free_list(list);
    return ADAMW_OK;
}

int adamw_list_set_hparams(adamw_list* list, double beta1, double beta2, double eps)
{
    osr::clear_error();
    if (!list)
        return fail(ADAMW_EINVAL, "list is NULL");
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) ||
        !(eps >= 0.0 && std::isfinite(eps)))
        return fail(ADAMW_EINVAL, "need 0 <= beta1, beta2 < 1 and finite eps >= 0");
    list->beta1 = beta1;
    list->beta2 = beta2;
    list->eps = eps;
    return ADAMW_OK;
}

int adamw_list_set_decay(adamw_list* list, const uint8_t* decay, int32_t n_tensors)
{
    osr::clear_error();
    if (!list)
        return fail(ADAMW_EINVAL, "list is NULL");
    if (decay && n_tensors != int32_t(list->numels.size()))
        return fail(ADAMW_EINVAL, "n_tensors=%d, the list has %d tensors", n_tensors,
                    int32_t(list->numels.size()));
    for (size_t k = 0; k < list->tensors.size(); ++k) {
        list->decay[k] = !decay || decay[k] ? 1 : 0;
        uint32_t& f = list->tensors[k].flags;
        f = list->decay[k] ? f | osr::kListDecay : f & ~osr::kListDecay;
    }
    return list->bound ? upload(list) : ADAMW_OK;
}

int adamw_list_bind(adamw_list* list, float* const* d_w, void* const* d_g, int32_t g_dtype,
                    void* const* d_m, void* const* d_v, float* const* d_m_scale,
                    float* const* d_v_scale, void* const* d_w_lp, int32_t w_lp_dtype)
{
    osr::clear_error();
    if (!list)
        return fail(ADAMW_EINVAL, "list is NULL");
    if (!list->numels.empty() && (!d_w || !d_g || !d_m || !d_v))
        return fail(ADAMW_EINVAL, "d_w, d_g, d_m or d_v is NULL");
    if (g_dtype != ADAMW_DTYPE_F32 && g_dtype != ADAMW_DTYPE_BF16 && g_dtype != ADAMW_DTYPE_F16)
        return fail(ADAMW_EINVAL, "g_dtype=%d is not F32, BF16 or F16", g_dtype);
    if (d_w_lp && w_lp_dtype != ADAMW_DTYPE_BF16 && w_lp_dtype != ADAMW_DTYPE_F16)
        return fail(ADAMW_EINVAL, "w_lp_dtype=%d is not BF16 or F16", w_lp_dtype);
    try {
        return bind_list(list, d_w, d_g, g_dtype, d_m, d_v, d_m_scale, d_v_scale, d_w_lp,
                         w_lp_dtype);
    } catch (const std::bad_alloc&) {
        return fail(ADAMW_EINVAL, "out of host memory");
    }
}

int adamw_list_step(adamw_list* list, int32_t t, double lr, double wd, double clip,
                    double grad_scale, uint32_t seed, int32_t flags, void* stream)
{
    osr::clear_error();
    if (!list)
        return fail(ADAMW_EINVAL, "list is NULL");
    if (!list->bound)
        return fail(ADAMW_ESTATE, "no arrays are bound to the list");
    if (t < 1)
        return fail(ADAMW_EINVAL, "t=%d: the first update has t = 1", t);
    if (!(lr >= 0.0 && std::isfinite(lr)) || !(wd >= 0.0 && std::isfinite(wd)))
        return fail(ADAMW_EINVAL, "lr=%g wd=%g must be finite and >= 0", lr, wd);
    if (!(clip > 0.0))
        return fail(ADAMW_EINVAL, "clip=%g must be > 0 (INFINITY disables clipping)", clip);
    if (!(grad_scale > 0.0 && std::isfinite(grad_scale)))
        return fail(ADAMW_EINVAL, "grad_scale=%g must be finite and > 0", grad_scale);
    if (flags & ~ADAMW_ZERO_GRAD)
        return fail(ADAMW_EINVAL, "unknown flags 0x%x", flags);
    DeviceScope scope(list->device);
    osr::StepScalars k = osr::step_scalars(list->beta1, list->beta2, list->eps, t, lr, wd);
    k.chunk_ctr = list->d_counters();
    k.fin = osr::NormFinish{list->d_partials(), osr::list_norm_blocks(list->n_units), clip,
                            grad_scale,         list->d_res(),
                            list->h_res_dev};
    const osr::ListView view{list->d_tensors, list->d_units, list->n_units};
    const osr::ListView plain{list->d_tensors, list->d_units, list->n_plain};
    const osr::ListView eight{list->d_tensors, list->d_units + list->n_plain,
                              list->n_units - list->n_plain};
    int e = osr::launch_list_norm(view, list->g_dtype, list->d_partials(), stream);
    if (e == cudaSuccess)
        e = osr::launch_list_step(plain, eight, list->g_dtype, list->w_lp_dtype, k,
                                  osr::rounding_key(seed, t), (flags & ADAMW_ZERO_GRAD) != 0,
                                  list->most, stream);
    if (e != cudaSuccess)
        return cuda_fail(cudaError_t(e), "list step launch");
    // for adamw_list_last_norm; a captured step is not one the host can wait for
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    CUDA_TRY(cudaStreamIsCapturing(st, &cap));
    if (cap == cudaStreamCaptureStatusNone) {
        CUDA_TRY(cudaEventRecord(list->ev_norm, st));
        list->launched = true;
    }
    return ADAMW_OK;
}

int adamw_list_last_norm(adamw_list* list, double* norm_out, float* scale_out)
{
    osr::clear_error();
    if (!list)
        return fail(ADAMW_EINVAL, "list is NULL");
    if (!list->launched)
        return fail(ADAMW_ESTATE, "no step has run on this list");
    CUDA_TRY(cudaEventSynchronize(list->ev_norm));
    volatile osr::NormResult* r = list->h_res;
    const double norm = r->norm;
    if (norm_out)
        *norm_out = norm;
    if (scale_out)
        *scale_out = r->scale;
    if (r->nonfinite)
        return fail(ADAMW_ENONFINITE, "gradient norm is %g: the update was skipped", norm);
    return ADAMW_OK;
}

}  // extern "C"
