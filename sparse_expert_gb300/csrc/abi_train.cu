// C ABI of the training-step operators: argument checks and launches.  As in
// the layer's entry points, arguments are validated on the host before any
// CUDA call, so an argument error enqueues nothing.
#include <cmath>
#include <cstring>

#include "moe_gb300.h"
#include "internal.h"

using namespace moe;

namespace {

// The last-error text is a std::string: if even that cannot be had, the
// status alone is returned, and nothing is thrown through the C boundary.
moe_status_t fail(moe_status_t s, const char* msg) noexcept {
  try {
    set_last_error(msg);
  } catch (...) {
  }
  return s;
}

moe_status_t cuda_fail(cudaError_t e, const char* where) noexcept {
  try {
    set_last_error(std::string(where) + ": " + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) + ")");
  } catch (...) {
  }
  return MOE_ERR_CUDA;
}

moe_status_t device_info(DeviceInfo* info) noexcept {
  const cudaError_t e = current_device_info(info);
  if (e == cudaErrorNoDevice || e == cudaErrorInsufficientDriver)
    return fail(MOE_ERR_NO_DEVICE, "no CUDA device available");
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  if (info->cc_major != 10 || info->cc_minor != 3)
    return fail(MOE_ERR_NO_DEVICE, "the library is built for sm_103a (GB300)");
  return MOE_OK;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool known(int32_t dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }
size_t size_of(int32_t dtype) { return dtype == MOE_F32 ? 4 : 2; }

moe_status_t check_norm(int64_t T, int32_t d, int32_t dtype, int32_t weight_dtype) {
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T must not be negative");
  if (T >= (int64_t(1) << 31)) return fail(MOE_ERR_UNSUPPORTED, "T must be below 2^31");
  if (d < 1 || d > 65536) return fail(MOE_ERR_UNSUPPORTED, "d must be in [1, 65536]");
  if (!known(dtype)) return fail(MOE_ERR_UNSUPPORTED, "dtype must be MOE_F32, MOE_BF16 or MOE_F16");
  if (weight_dtype != MOE_F32 && weight_dtype != dtype)
    return fail(MOE_ERR_UNSUPPORTED, "weight_dtype must be MOE_F32 or the rows' dtype");
  return MOE_OK;
}

// Rows given by the caller: present, aligned to their element, apart.
moe_status_t check_rows(const void* p, int64_t stride, int64_t T, int32_t d, int32_t dtype, const char* what) {
  if (!p) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(p, size_of(dtype))) return fail(MOE_ERR_INVALID_ARG, "rows must be aligned to their element size");
  if (T > 1 && stride < d) return fail(MOE_ERR_INVALID_ARG, what);
  return MOE_OK;
}

moe_status_t check_list(const moe_adamw_tensor_t* tensors, int32_t n_tensors, bool states) {
  if (n_tensors < 0) return fail(MOE_ERR_INVALID_ARG, "n_tensors must not be negative");
  if (n_tensors > 0 && !tensors) return fail(MOE_ERR_INVALID_ARG, "NULL tensor list");
  for (int32_t i = 0; i < n_tensors; ++i) {
    const moe_adamw_tensor_t& t = tensors[i];
    if (t.n < 0) return fail(MOE_ERR_INVALID_ARG, "a tensor's n must not be negative");
    if (t.n > kTensorMaxValues) return fail(MOE_ERR_UNSUPPORTED, "a tensor's n must be at most 2^42 - 2048");
    if (!known(t.grad_type)) return fail(MOE_ERR_UNSUPPORTED, "grad_type must be MOE_F32, MOE_BF16 or MOE_F16");
    if (t.n == 0) continue;
    if (!t.grad) return fail(MOE_ERR_INVALID_ARG, "NULL gradient");
    if (!aligned(t.grad, size_of(t.grad_type)))
      return fail(MOE_ERR_INVALID_ARG, "a gradient must be aligned to its element size");
    if (!states) continue;
    if (!known(t.param_type)) return fail(MOE_ERR_UNSUPPORTED, "param_type must be MOE_F32, MOE_BF16 or MOE_F16");
    if (t.state_bits != 32 && t.state_bits != 8) return fail(MOE_ERR_UNSUPPORTED, "state_bits must be 32 or 8");
    if (!t.param || !t.m || !t.v) return fail(MOE_ERR_INVALID_ARG, "NULL parameter or state");
    if (t.state_bits == 8 && (!t.m_scale || !t.v_scale))
      return fail(MOE_ERR_INVALID_ARG, "8-bit states need m_scale and v_scale");
    if (!std::isfinite(t.decay) || t.decay < 0.0f)
      return fail(MOE_ERR_INVALID_ARG, "decay must be finite and not negative");
    if (!aligned(t.param, size_of(t.param_type)) || !aligned(t.master, 4) || !aligned(t.m_scale, 4) ||
        !aligned(t.v_scale, 4) || (t.state_bits == 32 && (!aligned(t.m, 4) || !aligned(t.v, 4))))
      return fail(MOE_ERR_INVALID_ARG, "parameters, masters and states must be aligned to their element size");
  }
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_layer_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                            const void* weight, const void* bias, int64_t T, int32_t d, int32_t dtype,
                            int32_t weight_dtype, float eps, void* y, void* z, float* stats, moe_stream_t stream) {
  moe_status_t s = check_norm(T, d, dtype, weight_dtype);
  if (s != MOE_OK) return s;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(MOE_ERR_INVALID_ARG, "eps must be finite and not negative");
  if ((residual != nullptr) != (z != nullptr) && T > 0)
    return fail(MOE_ERR_INVALID_ARG, "z is written with a residual, and only then");
  if (T == 0) return MOE_OK;
  if ((s = check_rows(x, x_stride, T, d, dtype, "x_stride must be at least d")) != MOE_OK) return s;
  if (residual &&
      (s = check_rows(residual, residual_stride, T, d, dtype, "residual_stride must be at least d")) != MOE_OK)
    return s;
  if (!y || !stats) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(y, size_of(dtype)) || !aligned(z, size_of(dtype)) || !aligned(stats, 4) ||
      !aligned(weight, size_of(weight_dtype)) || !aligned(bias, size_of(weight_dtype)))
    return fail(MOE_ERR_INVALID_ARG, "y, z, stats, weight and bias must be aligned to their element size");
  DeviceInfo dev;
  if ((s = device_info(&dev)) != MOE_OK) return s;
  const cudaError_t e = launch_layer_norm(NormForward{x, x_stride, residual, residual_stride, weight, bias, T, d, dtype,
                                                      weight_dtype, eps, y, z, stats},
                                          dev.num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "layer norm launch");
}

size_t moe_layer_norm_backward_workspace_bytes(int64_t T, int32_t d) {
  if (T < 0 || d < 1) return 0;
  return norm_backward_workspace_bytes(T, d);
}

moe_status_t moe_layer_norm_backward(const void* dy, int64_t dy_stride, const void* z, int64_t z_stride,
                                     const float* stats, const void* weight, const void* dz, int64_t dz_stride,
                                     int64_t T, int32_t d, int32_t dtype, int32_t weight_dtype, void* dx,
                                     float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                                     moe_stream_t stream) {
  moe_status_t s = check_norm(T, d, dtype, weight_dtype);
  if (s != MOE_OK) return s;
  if (!aligned(dweight, 4) || !aligned(dbias, 4))
    return fail(MOE_ERR_INVALID_ARG, "dweight and dbias must be aligned to their element size");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  if (T == 0) {
    if (!dweight && !dbias) return MOE_OK;
    if ((s = device_info(&dev)) != MOE_OK) return s;
    for (float* sum : {dweight, dbias}) {
      if (!sum) continue;
      const cudaError_t e = cudaMemsetAsync(sum, 0, static_cast<size_t>(d) * 4, st);
      if (e != cudaSuccess) return cuda_fail(e, "gradient clear");
    }
    return MOE_OK;
  }
  if ((s = check_rows(dy, dy_stride, T, d, dtype, "dy_stride must be at least d")) != MOE_OK) return s;
  if ((s = check_rows(z, z_stride, T, d, dtype, "z_stride must be at least d")) != MOE_OK) return s;
  if (dz && (s = check_rows(dz, dz_stride, T, d, dtype, "dz_stride must be at least d")) != MOE_OK) return s;
  if (!stats || !dx) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(stats, 4) || !aligned(dx, size_of(dtype)) || !aligned(weight, size_of(weight_dtype)))
    return fail(MOE_ERR_INVALID_ARG, "stats, dx and weight must be aligned to their element size");
  if ((dweight || dbias) && (!workspace || workspace_bytes < norm_backward_workspace_bytes(T, d) ||
                             !aligned(workspace, kAlign)))
    return fail(MOE_ERR_WORKSPACE,
                "the workspace must hold moe_layer_norm_backward_workspace_bytes, 256-byte aligned");
  if ((s = device_info(&dev)) != MOE_OK) return s;
  const cudaError_t e = launch_layer_norm_backward(
      NormBackward{dy, dy_stride, z, z_stride, stats, weight, dz, dz_stride, T, d, dtype, weight_dtype, dx, dweight,
                   dbias, static_cast<float*>(workspace)},
      dev.num_sms, st);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "layer norm backward launch");
}

size_t moe_router_loss_workspace_bytes(void) { return router_loss_workspace_bytes(); }

moe_status_t moe_router_loss(const float* logits, const int32_t* counts, const uint8_t* mask, int64_t T, int32_t E,
                             float balance_coef, float z_coef, const float* d_in, float* d_logits, float* losses,
                             void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T must not be negative");
  if (E < 1 || E > MOE_MAX_EXPERTS) return fail(MOE_ERR_UNSUPPORTED, "E must be in [1, 1024]");
  if (T >= (int64_t(1) << 40) / E) return fail(MOE_ERR_UNSUPPORTED, "T*E must be below 2^40");
  if (!std::isfinite(balance_coef) || !std::isfinite(z_coef))
    return fail(MOE_ERR_INVALID_ARG, "the coefficients must be finite");
  if (!losses || !aligned(losses, 4)) return fail(MOE_ERR_INVALID_ARG, "losses is NULL or misaligned");
  DeviceInfo dev;
  moe_status_t s;
  if (T == 0) {
    if ((s = device_info(&dev)) != MOE_OK) return s;
    const cudaError_t e = cudaMemsetAsync(losses, 0, 8, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "losses clear");
  }
  if (!logits || !counts || !d_logits) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(logits, 4) || !aligned(counts, 4) || !aligned(d_in, 4) || !aligned(d_logits, 4))
    return fail(MOE_ERR_INVALID_ARG, "logits, counts and gradients must be 4-byte aligned");
  if (!workspace || workspace_bytes < router_loss_workspace_bytes() || !aligned(workspace, kAlign))
    return fail(MOE_ERR_WORKSPACE, "the workspace must hold moe_router_loss_workspace_bytes, 256-byte aligned");
  if ((s = device_info(&dev)) != MOE_OK) return s;
  const cudaError_t e = launch_router_loss(RouterLoss{logits, counts, mask, T, E, balance_coef, z_coef, d_in, d_logits,
                                                      losses, workspace},
                                           dev.num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "router loss launch");
}

moe_status_t moe_adamw_hyper(double lr, double beta1, double beta2, double eps, double weight_decay, int64_t step,
                             moe_adamw_hyper_t* hyper) {
  if (!hyper) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!(lr >= 0.0) || !(eps >= 0.0) || !(weight_decay >= 0.0) || !std::isfinite(lr) || !std::isfinite(eps) ||
      !std::isfinite(weight_decay))
    return fail(MOE_ERR_INVALID_ARG, "lr, eps and weight_decay must be finite and not negative");
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0))
    return fail(MOE_ERR_INVALID_ARG, "beta1 and beta2 must be in [0, 1)");
  if (step < 1) return fail(MOE_ERR_INVALID_ARG, "step must be at least 1");
  hyper->beta1 = static_cast<float>(beta1);
  hyper->one_minus_beta1 = static_cast<float>(1.0 - beta1);
  hyper->beta2 = static_cast<float>(beta2);
  hyper->one_minus_beta2 = static_cast<float>(1.0 - beta2);
  const double t = static_cast<double>(step);
  hyper->step_size = static_cast<float>(lr / (1.0 - std::pow(beta1, t)));
  hyper->decay = static_cast<float>(lr * weight_decay);
  hyper->inv_sqrt_bias = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, t)));
  hyper->eps = static_cast<float>(eps);
  return MOE_OK;
}

moe_status_t moe_adamw_step(const moe_adamw_tensor_t* tensors, int32_t n_tensors, const moe_adamw_hyper_t* hyper,
                            const moe_adamw_hyper_t* hyper_dev, const float* grad_scale, moe_stream_t stream) {
  moe_status_t s = check_list(tensors, n_tensors, true);
  if (s != MOE_OK) return s;
  if ((hyper != nullptr) == (hyper_dev != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "exactly one of hyper and hyper_dev must be given");
  if (!aligned(hyper_dev, 4) || !aligned(grad_scale, 4))
    return fail(MOE_ERR_INVALID_ARG, "hyper_dev and grad_scale must be 4-byte aligned");
  DeviceInfo dev;
  if ((s = device_info(&dev)) != MOE_OK) return s;
  const cudaError_t e =
      launch_adamw(tensors, n_tensors, hyper, hyper_dev, grad_scale, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "AdamW launch");
}

size_t moe_grad_norm_workspace_bytes(void) { return grad_norm_workspace_bytes(); }

moe_status_t moe_grad_norm(const moe_adamw_tensor_t* tensors, int32_t n_tensors, float max_norm, float* out,
                           void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (n_tensors > kGradNormMaxTensors)
    return fail(MOE_ERR_UNSUPPORTED, "n_tensors must be at most 1,572,864 for the gradient norm");
  moe_status_t s = check_list(tensors, n_tensors, false);
  if (s != MOE_OK) return s;
  if (!(max_norm > 0.0f)) return fail(MOE_ERR_INVALID_ARG, "max_norm must be positive (infinity: no clipping)");
  if (!out || !aligned(out, 4)) return fail(MOE_ERR_INVALID_ARG, "out is NULL or misaligned");
  if (!workspace || workspace_bytes < grad_norm_workspace_bytes() || !aligned(workspace, kAlign))
    return fail(MOE_ERR_WORKSPACE, "the workspace must hold moe_grad_norm_workspace_bytes, 256-byte aligned");
  DeviceInfo dev;
  if ((s = device_info(&dev)) != MOE_OK) return s;
  const cudaError_t e = launch_grad_norm(tensors, n_tensors, max_norm, out, static_cast<double*>(workspace),
                                         dev.num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "gradient norm launch");
}

}  // extern "C"
