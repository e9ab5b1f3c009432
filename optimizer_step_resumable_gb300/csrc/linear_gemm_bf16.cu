// linear_gemm_bf16.cu -- products whose output is bfloat16.
#include "linear_gemm.cuh"

namespace osr {

int linear_store_bf16(int bn, const StoreProduct& p, bool plain, bool bf16, int sm_count,
                      void* stream)
{
    return plain ? detail::store_one<ADAMW_DTYPE_BF16, true>(bn, p, bf16, sm_count, stream)
                 : detail::store_one<ADAMW_DTYPE_BF16, false>(bn, p, bf16, sm_count, stream);
}

}  // namespace osr
