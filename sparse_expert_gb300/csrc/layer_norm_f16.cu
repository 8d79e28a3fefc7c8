// Layer norm of fp16 rows.
#include "layer_norm_backward.cuh"
#include "layer_norm_forward.cuh"

namespace moe {

template cudaError_t norm_forward_typed<__half>(NormForwardArgs&, int, cudaStream_t);
template cudaError_t norm_backward_typed<__half>(NormBackwardArgs&, int, int*, cudaStream_t);

}  // namespace moe
