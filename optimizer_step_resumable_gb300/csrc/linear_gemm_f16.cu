// linear_gemm_f16.cu -- products whose output is binary16.
#include "linear_gemm.cuh"

namespace osr {

int linear_store_f16(int bn, const StoreProduct& p, bool plain, bool bf16, int sm_count,
                     void* stream)
{
    return plain ? detail::store_one<ADAMW_DTYPE_F16, true>(bn, p, bf16, sm_count, stream)
                 : detail::store_one<ADAMW_DTYPE_F16, false>(bn, p, bf16, sm_count, stream);
}

}  // namespace osr
