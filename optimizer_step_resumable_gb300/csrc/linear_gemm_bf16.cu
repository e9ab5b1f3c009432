// linear_gemm_bf16.cu -- products whose output is bfloat16.
#include "linear_gemm.cuh"

namespace osr {

int linear_store_bf16(int bn, const GemmOperand& a, const GemmOperand& b, const GemmShape& s,
                      bool bf16, const StoreParams& p, int sm_count, void* stream)
{
    return detail::linear_store<ADAMW_DTYPE_BF16>(bn, a, b, s, bf16, p, sm_count, stream);
}

}  // namespace osr
