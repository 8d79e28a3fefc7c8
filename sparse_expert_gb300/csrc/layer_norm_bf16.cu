// Layer norm of bf16 rows.
#include "layer_norm_backward.cuh"
#include "layer_norm_forward.cuh"

namespace moe {

template cudaError_t norm_forward_typed<__nv_bfloat16>(NormForwardArgs&, int, cudaStream_t);
template cudaError_t norm_backward_typed<__nv_bfloat16>(NormBackwardArgs&, int, int*, cudaStream_t);

}  // namespace moe
