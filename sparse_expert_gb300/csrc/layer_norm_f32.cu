// Layer norm of fp32 rows.
#include "layer_norm_backward.cuh"
#include "layer_norm_forward.cuh"

namespace moe {

template cudaError_t norm_forward_typed<float>(NormForwardArgs&, int, cudaStream_t);
template cudaError_t norm_backward_typed<float>(NormBackwardArgs&, int, int*, cudaStream_t);

}  // namespace moe
