// linear_gemm_two_f16.cu -- two products in a launch, the first one's output
// binary16.
#include "linear_gemm.cuh"

namespace osr {

int linear_store_two_f16(const StoreProduct& p, const StoreProduct& q, const GemmDeal& deal,
                         void* stream)
{
    constexpr bool bf16 = false;
    return q.p.o.dtype == ADAMW_DTYPE_F32
               ? detail::store_two<ADAMW_DTYPE_F16, ADAMW_DTYPE_F32>(p, q, bf16, deal, stream)
               : detail::store_two<ADAMW_DTYPE_F16, ADAMW_DTYPE_F16>(p, q, bf16, deal, stream);
}

}  // namespace osr
