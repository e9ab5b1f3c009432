// linear_gemm_two_f32.cu -- two products in a launch, the first one's output
// float32.
#include "linear_gemm.cuh"

namespace osr {

int linear_store_two_f32(const StoreProduct& p, const StoreProduct& q, bool bf16,
                         const GemmDeal& deal, void* stream)
{
    switch (q.p.o.dtype) {
    case ADAMW_DTYPE_F32:
        return detail::store_two<ADAMW_DTYPE_F32, ADAMW_DTYPE_F32>(p, q, bf16, deal, stream);
    case ADAMW_DTYPE_BF16:
        return detail::store_two<ADAMW_DTYPE_F32, ADAMW_DTYPE_BF16>(p, q, bf16, deal, stream);
    default: return detail::store_two<ADAMW_DTYPE_F32, ADAMW_DTYPE_F16>(p, q, bf16, deal, stream);
    }
}

}  // namespace osr
