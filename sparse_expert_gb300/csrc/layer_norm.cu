// Layer norm: the launches by element type, and the last step of the
// backward's column sums (the formulas and the forms: layer_norm.cuh).
#include "layer_norm.cuh"

namespace moe {
namespace {

// dw and db: the blocks' sums added in block order, in 32 interleaved
// partial sums a column, each a warp's: a read of [blocks][2][d] fp32 that
// still lies in L2, bound by its latency and that of the launch, which is
// made while the rows' kernel runs (152 blocks of 6,144 columns, 7.5 MB:
// 6-8 us behind a rows' kernel of 119 us).
__global__ void __launch_bounds__(1024) finish_kernel(const float* __restrict__ partial, int blocks, int d,
                                                      float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float part[32][33];
  wait_for_previous();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? db : dw;
  if (out == nullptr) return;
  float s = 0.0f;
  if (j < d)
    for (int b = slice; b < blocks; b += 32) s += partial[(static_cast<int64_t>(b) * 2 + blockIdx.y) * d + j];
  part[slice][lane] = s;
  __syncthreads();
  s = warp_sum(part[lane][slice]);  // column `slice` of the block
  const int col = blockIdx.x * 32 + slice;
  if (lane == 0 && col < d) out[col] = s;
}

}  // namespace

cudaError_t launch_layer_norm(const NormForward& f, int num_sms, cudaStream_t stream) {
  NormForwardArgs a{{f.x, f.x_stride}, {f.residual, f.residual_stride}, f.weight, f.bias, f.weight_dtype == MOE_F32,
                    f.T, f.d, f.eps, f.y, f.z, f.stats, 0, 0, 0, false};
  switch (f.dtype) {
    case MOE_F32: return norm_forward_typed<float>(a, num_sms, stream);
    case MOE_BF16: return norm_forward_typed<__nv_bfloat16>(a, num_sms, stream);
    default: return norm_forward_typed<__half>(a, num_sms, stream);
  }
}

size_t norm_backward_workspace_bytes(int64_t T, int d) {
  const int64_t blocks = T < kNormMaxBlocks ? T : kNormMaxBlocks;
  return align_up(static_cast<size_t>(blocks < 1 ? 1 : blocks) * 2 * d * 4);
}

cudaError_t launch_layer_norm_backward(const NormBackward& f, int num_sms, cudaStream_t stream) {
  NormBackwardArgs a{{f.dy, f.dy_stride}, {f.z, f.z_stride}, {f.dz, f.dz_stride}, f.stats, f.weight,
                     f.weight_dtype == MOE_F32, f.T, f.d, f.dx, f.partial, f.dweight, f.dbias, f.dweight != nullptr,
                     f.dbias != nullptr, 0, 0};
  int blocks = 0;
  cudaError_t err;
  switch (f.dtype) {
    case MOE_F32: err = norm_backward_typed<float>(a, num_sms, &blocks, stream); break;
    case MOE_BF16: err = norm_backward_typed<__nv_bfloat16>(a, num_sms, &blocks, stream); break;
    default: err = norm_backward_typed<__half>(a, num_sms, &blocks, stream); break;
  }
  if (err != cudaSuccess || a.cluster || !(a.want_w || a.want_b)) return err;
  return launch_dependent(finish_kernel, dim3((f.d + 31) / 32, 2), 1024, 0, stream, f.partial, blocks, f.d, f.dweight,
                          f.dbias);
}

}  // namespace moe
