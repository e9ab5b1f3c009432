// layernorm_bwd_f32.cu -- the layer norm's backward pass for f32 rows.
#include "layernorm_bwd.cuh"

namespace osr {

template int launch_ln_backward_typed<float>(const LnBackward&, int, std::atomic<int>*, int32_t*,
                                             cudaStream_t);

}  // namespace osr
