// layernorm_bwd_bf16.cu -- the layer norm's backward pass for bf16 rows.
#include "layernorm_bwd.cuh"

namespace osr {

template int launch_ln_backward_typed<__nv_bfloat16>(const LnBackward&, int, std::atomic<int>*, int32_t*,
                                             cudaStream_t);

}  // namespace osr
