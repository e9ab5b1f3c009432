// layernorm_bwd_f16.cu -- the layer norm's backward pass for f16 rows.
#include "layernorm_bwd.cuh"

namespace osr {

template int launch_ln_backward_typed<__half>(const LnBackward&, int, std::atomic<int>*, int32_t*,
                                             cudaStream_t);

}  // namespace osr
