// linear_gemm_two_bf16.cu -- two products in a launch, the first one's output
// bfloat16.
#include "linear_gemm.cuh"

namespace osr {

int linear_store_two_bf16(const StoreProduct& p, const StoreProduct& q, const GemmDeal& deal,
                          void* stream)
{
    constexpr bool bf16 = true;
    return q.p.o.dtype == ADAMW_DTYPE_F32
               ? detail::store_two<ADAMW_DTYPE_BF16, ADAMW_DTYPE_F32>(p, q, bf16, deal, stream)
               : detail::store_two<ADAMW_DTYPE_BF16, ADAMW_DTYPE_BF16>(p, q, bf16, deal, stream);
}

}  // namespace osr
