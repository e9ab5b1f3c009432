// linear_gemm_f32.cu -- products whose output is float32.
#include "linear_gemm.cuh"

namespace osr {

int linear_store_f32(int bn, const StoreProduct& p, bool bf16, int sm_count, void* stream)
{
    return detail::store_one<ADAMW_DTYPE_F32, true>(bn, p, bf16, sm_count, stream);
}

}  // namespace osr
