// C ABI of the layer for a few tokens and of 4-bit weights: argument checks,
// workspace layout and launches.  As everywhere, arguments are validated on
// the host before any CUDA call.
#include "moe_gb300.h"
#include "few.cuh"
#include "int4.cuh"
#include "internal.h"

using namespace moe;

namespace {

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

bool known_group(int32_t group) { return group == 32 || group == 64 || group == 128; }

// Sizes of the layer for a few tokens, without the weights' own.
moe_status_t check_few(int64_t T, int32_t E, int32_t k, int32_t d, int32_t f) {
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T must be >= 0");
  if (T > MOE_FEW_MAX_TOKENS) return fail(MOE_ERR_UNSUPPORTED, "T must be at most MOE_FEW_MAX_TOKENS (64)");
  if (E < 1 || E > MOE_MAX_EXPERTS) return fail(MOE_ERR_UNSUPPORTED, "E must be in [1, 1024]");
  if (k < 1 || k > E || k > MOE_MAX_TOPK) return fail(MOE_ERR_UNSUPPORTED, "k must be in [1, min(E, 32)]");
  if (d < 64 || d > 65536 || d % 64 != 0) return fail(MOE_ERR_UNSUPPORTED, "d must be a multiple of 64 in [64, 65536]");
  if (f < 64 || f > 65536 || f % 64 != 0) return fail(MOE_ERR_UNSUPPORTED, "f must be a multiple of 64 in [64, 65536]");
  return MOE_OK;
}

moe_status_t check_int4_experts(int32_t E, int32_t d, int32_t f, int32_t group) {
  if (E < 1 || E > MOE_MAX_EXPERTS) return fail(MOE_ERR_UNSUPPORTED, "E must be in [1, 1024]");
  if (d < 128 || d > 65536 || d % 128 != 0 || f < 128 || f > 65536 || f % 128 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "4-bit expert weights need d and f multiples of 128 in [128, 65536]");
  if (!known_group(group)) return fail(MOE_ERR_UNSUPPORTED, "group must be 32, 64 or 128");
  return MOE_OK;
}

moe_status_t check_int4_matrix(int64_t K, int64_t N, int32_t group) {
  if (K < 8 || K > 65536 || K % 8 != 0) return fail(MOE_ERR_UNSUPPORTED, "K must be a multiple of 8 in [8, 65536]");
  if (N < 1 || N > (int64_t(1) << 24)) return fail(MOE_ERR_UNSUPPORTED, "N must be in [1, 2^24]");
  if (!known_group(group)) return fail(MOE_ERR_UNSUPPORTED, "group must be 32, 64 or 128");
  return MOE_OK;
}

struct FewLayout {
  size_t counters, units, pair_row, topk_idx, topk_w, logits, h, y, total;
  int n_counters;
};

FewLayout few_layout(int64_t T, int32_t E, int32_t k, int32_t d, int32_t f) {
  const size_t P = static_cast<size_t>(T) * k;
  FewLayout L{};
  size_t o = sizeof(FewHeader);
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  L.n_counters = static_cast<int>(P) + (d + kFewStrip - 1) / kFewStrip;  // units, at most one a pair; output strips
  L.counters = take(sizeof(int32_t) * L.n_counters);
  L.units = take(sizeof(FewUnit) * P);
  L.pair_row = take(sizeof(int32_t) * P);
  L.topk_idx = take(sizeof(int32_t) * P);
  L.topk_w = take(sizeof(float) * P);
  L.logits = take(sizeof(float) * static_cast<size_t>(T) * E);
  L.h = take(size_t(4) * P * f);  // high parts, then low parts
  L.y = take(sizeof(float) * P * d);
  L.total = o;
  return L;
}

// spoiled (of a check of the waits, else -1): a counter of finished pieces that
// is set to what no number of pieces makes it.
moe_status_t few(const void* x, const float* logits, const void* router, const void* packed, int32_t weights,
                 int32_t group, int64_t T, int32_t d, int32_t E, int32_t k, int32_t f, int32_t renormalize, void* out,
                 int32_t* topk_idx_out, float* topk_w_out, void* workspace, size_t workspace_bytes,
                 moe_stream_t stream, int64_t spoiled = -1, uint64_t wait_ns = kWaitLimitNs) {
  moe_status_t s = check_few(T, E, k, d, f);
  if (s != MOE_OK) return s;
  switch (weights) {
    case MOE_WEIGHTS_BF16:
      break;
    case MOE_WEIGHTS_FP8:
      if (d % 128 != 0 || f % 128 != 0)
        return fail(MOE_ERR_UNSUPPORTED, "FP8 expert weights need d and f multiples of 128");
      break;
    case MOE_WEIGHTS_INT4:
      if ((s = check_int4_experts(E, d, f, group)) != MOE_OK) return s;
      break;
    default:
      return fail(MOE_ERR_UNSUPPORTED, "weights must be MOE_WEIGHTS_BF16, MOE_WEIGHTS_FP8 or MOE_WEIGHTS_INT4");
  }
  if (router && E > 512) return fail(MOE_ERR_UNSUPPORTED, "the fused router takes E <= 512");
  if (!packed) return fail(MOE_ERR_INVALID_ARG, "NULL packed weights");
  if (T > 0 && (!x || (!logits && !router) || !out)) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(router, 16) || !aligned(logits, 4))
    return fail(MOE_ERR_INVALID_ARG, "x, out and the router weights must be 16-byte aligned, logits 4-byte");
  if (!aligned(packed, weights == MOE_WEIGHTS_BF16 ? 16 : kAlign))
    return fail(MOE_ERR_INVALID_ARG, "packed weights must be aligned to 16 bytes (bf16) or 256 bytes (FP8, 4 bits)");
  if (!aligned(topk_idx_out, 4) || !aligned(topk_w_out, 4))
    return fail(MOE_ERR_INVALID_ARG, "topk_idx_out and topk_w_out must be 4-byte aligned");
  const FewLayout L = few_layout(T, E, k, d, f);
  if (!workspace || workspace_bytes < L.total || !aligned(workspace, kAlign))
    return fail(MOE_ERR_WORKSPACE, "workspace needs moe_forward_few_workspace_bytes bytes, 256-byte aligned");
  DeviceInfo dev;
  if ((s = device_info(&dev)) != MOE_OK) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (T == 0) {
    const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(FewHeader), st);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "workspace clear");
  }
  auto* counters = reinterpret_cast<int32_t*>(ws + L.counters);
  FewRoute r{};
  r.x = x;
  r.router = router;
  r.logits = logits;
  r.logits_out = reinterpret_cast<float*>(ws + L.logits);
  r.T = static_cast<int>(T);
  r.d = d;
  r.E = E;
  r.E_pad = router_e_pad(E);
  r.k = k;
  r.renormalize = renormalize;
  r.topk_idx = topk_idx_out ? topk_idx_out : reinterpret_cast<int32_t*>(ws + L.topk_idx);
  r.topk_w = topk_w_out ? topk_w_out : reinterpret_cast<float*>(ws + L.topk_w);
  r.pair_row = reinterpret_cast<int32_t*>(ws + L.pair_row);
  r.units = reinterpret_cast<FewUnit*>(ws + L.units);
  r.header = reinterpret_cast<FewHeader*>(ws);
  r.counters = counters;
  r.n_counters = L.n_counters;
  cudaError_t e = launch_few_route(r, st);
  if (e != cudaSuccess) return cuda_fail(e, "route launch");
  if (spoiled >= 0) {
    e = cudaMemsetAsync(counters + spoiled, 0x80, sizeof(int32_t), st);
    if (e != cudaSuccess) return cuda_fail(e, "counter");
  }
  FewExperts p{};
  p.x = x;
  p.packed = packed;
  p.weights = weights;
  p.group = group;
  p.T = r.T;
  p.d = d;
  p.E = E;
  p.k = k;
  p.f = f;
  p.units = r.units;
  p.header = r.header;
  p.ready = counters;
  p.strips = counters + T * k;
  p.topk_w = r.topk_w;
  p.pair_row = r.pair_row;
  p.h = ws + L.h;
  p.y = reinterpret_cast<float*>(ws + L.y);
  p.out = out;
  p.wait_ns = wait_ns;
  e = launch_few_experts(p, dev.num_sms, st);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "experts launch");
}

// row_strips: strips of outputs that rows of x are fetched for (fewer than there are: a check of the waits).
moe_status_t linear(const void* x, int64_t x_stride, const void* packed, int64_t M, int64_t K, int64_t N, int32_t group,
                    void* out, int64_t out_stride, moe_stream_t stream, int32_t row_strips = INT32_MAX,
                    uint64_t wait_ns = kWaitLimitNs) {
  if (M < 0) return fail(MOE_ERR_INVALID_ARG, "M must not be negative");
  if (M > MOE_LINEAR_INT4_MAX_ROWS) return fail(MOE_ERR_UNSUPPORTED, "M must be at most MOE_LINEAR_INT4_MAX_ROWS (16)");
  moe_status_t s = check_int4_matrix(K, N, group);
  if (s != MOE_OK || M == 0) return s;
  if (!x || !packed || !out) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  if (M > 1 && (x_stride < K || out_stride < N))
    return fail(MOE_ERR_INVALID_ARG, "x_stride must be at least K and out_stride at least N");
  if (!aligned(x, 16) || (M > 1 && x_stride % 8 != 0))
    return fail(MOE_ERR_INVALID_ARG, "rows of x must be 16-byte aligned");
  if (!aligned(packed, kAlign) || !aligned(out, 2))
    return fail(MOE_ERR_INVALID_ARG, "packed must be 256-byte aligned, out 2-byte");
  DeviceInfo dev;
  if ((s = device_info(&dev)) != MOE_OK) return s;
  const cudaError_t e =
      launch_linear_int4(LinearInt4{x, x_stride, packed, static_cast<int>(M), static_cast<int>(K), static_cast<int>(N),
                                    group, out, out_stride, wait_ns, row_strips},
                         dev.num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "linear launch");
}

}  // namespace

extern "C" {

size_t moe_forward_few_workspace_bytes(int64_t T, int32_t E, int32_t k, int32_t d, int32_t f) {
  if (check_few(T, E, k, d, f) != MOE_OK) return 0;
  return few_layout(T, E, k, d, f).total;
}

moe_status_t moe_forward_few(const void* x, const float* logits, const void* packed, int32_t weights, int32_t group,
                             int64_t T, int32_t d, int32_t E, int32_t k, int32_t f, int32_t renormalize, void* out,
                             int32_t* topk_idx_out, float* topk_w_out, void* workspace, size_t workspace_bytes,
                             moe_stream_t stream) {
  return few(x, logits, nullptr, packed, weights, group, T, d, E, k, f, renormalize, out, topk_idx_out, topk_w_out,
             workspace, workspace_bytes, stream);
}

moe_status_t moe_forward_few_routed(const void* x, const void* router_packed, const void* packed, int32_t weights,
                                    int32_t group, int64_t T, int32_t d, int32_t E, int32_t k, int32_t f,
                                    int32_t renormalize, void* out, int32_t* topk_idx_out, float* topk_w_out,
                                    void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (!router_packed) return fail(MOE_ERR_INVALID_ARG, "NULL router weights");
  return few(x, nullptr, router_packed, packed, weights, group, T, d, E, k, f, renormalize, out, topk_idx_out,
             topk_w_out, workspace, workspace_bytes, stream);
}

moe_status_t moe_quantize_int4(const void* w, int64_t matrices, int64_t K, int64_t N, int32_t group, uint8_t* codes,
                               void* scales, moe_stream_t stream) {
  if (matrices < 0) return fail(MOE_ERR_INVALID_ARG, "matrices must not be negative");
  if (matrices > (int64_t(1) << 16)) return fail(MOE_ERR_UNSUPPORTED, "matrices must be at most 65536");
  moe_status_t s = check_int4_matrix(K, N, group);
  if (s != MOE_OK || matrices == 0) return s;
  if (!w || !codes || !scales) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(w, 2) || !aligned(scales, 2)) return fail(MOE_ERR_INVALID_ARG, "w and scales must be 2-byte aligned");
  DeviceInfo dev;
  if ((s = device_info(&dev)) != MOE_OK) return s;
  const cudaError_t e =
      launch_quantize_int4(w, matrices, K, N, group, codes, scales, dev.num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "quantize launch");
}

size_t moe_int4_packed_weight_bytes(int32_t E, int32_t d, int32_t f, int32_t group) {
  if (check_int4_experts(E, d, f, group) != MOE_OK) return 0;
  return align_up(int4_matrix_bytes(E, d, 2 * static_cast<int64_t>(f), group)) + int4_matrix_bytes(E, f, d, group);
}

moe_status_t moe_pack_weights_int4(const uint8_t* gate_codes, const void* gate_scales, const uint8_t* up_codes,
                                   const void* up_scales, const uint8_t* down_codes, const void* down_scales,
                                   int32_t E, int32_t d, int32_t f, int32_t group, void* packed,
                                   moe_stream_t stream) {
  moe_status_t s = check_int4_experts(E, d, f, group);
  if (s != MOE_OK) return s;
  if (!gate_codes || !gate_scales || !up_codes || !up_scales || !down_codes || !down_scales || !packed)
    return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(gate_scales, 2) || !aligned(up_scales, 2) || !aligned(down_scales, 2) || !aligned(packed, kAlign))
    return fail(MOE_ERR_INVALID_ARG, "scales must be 2-byte aligned, packed 256-byte");
  DeviceInfo dev;
  if ((s = device_info(&dev)) != MOE_OK) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_pack_int4(gate_codes, gate_scales, up_codes, up_scales, E, d, f, group, packed, dev.num_sms, st);
  if (e == cudaSuccess)
    e = launch_pack_int4(down_codes, down_scales, nullptr, nullptr, E, f, d, group,
                         static_cast<char*>(packed) + align_up(int4_matrix_bytes(E, d, 2 * static_cast<int64_t>(f), group)),
                         dev.num_sms, st);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "pack launch");
}

size_t moe_linear_int4_packed_bytes(int64_t K, int64_t N, int32_t group) {
  return check_int4_matrix(K, N, group) == MOE_OK ? int4_matrix_bytes(1, static_cast<int>(K), N, group) : 0;
}

moe_status_t moe_pack_linear_int4(const uint8_t* codes, const void* scales, int64_t K, int64_t N, int32_t group,
                                  void* packed, moe_stream_t stream) {
  moe_status_t s = check_int4_matrix(K, N, group);
  if (s != MOE_OK) return s;
  if (!codes || !scales || !packed) return fail(MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(scales, 2) || !aligned(packed, kAlign))
    return fail(MOE_ERR_INVALID_ARG, "scales must be 2-byte aligned, packed 256-byte");
  DeviceInfo dev;
  if ((s = device_info(&dev)) != MOE_OK) return s;
  const cudaError_t e = launch_pack_int4(codes, scales, nullptr, nullptr, 1, static_cast<int>(K), static_cast<int>(N),
                                         group, packed, dev.num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MOE_OK : cuda_fail(e, "pack launch");
}

moe_status_t moe_linear_int4(const void* x, int64_t x_stride, const void* packed, int64_t M, int64_t K, int64_t N,
                             int32_t group, void* out, int64_t out_stride, moe_stream_t stream) {
  return linear(x, x_stride, packed, M, K, N, group, out, out_stride, stream);
}

moe_status_t moe_selftest_few_wait(const void* x, const float* logits, const void* packed, int32_t weights,
                                   int32_t group, int64_t T, int32_t d, int32_t E, int32_t k, int32_t f, void* out,
                                   void* workspace, size_t workspace_bytes, int64_t spoiled, int64_t limit_ns,
                                   moe_stream_t stream) {
  const moe_status_t s = check_few(T, E, k, d, f);
  if (s != MOE_OK) return s;
  if (limit_ns < 1 || limit_ns > static_cast<int64_t>(kWaitLimitNs))
    return fail(MOE_ERR_INVALID_ARG, "limit_ns must be in [1, 2e9]");
  if (spoiled < -1 || spoiled >= few_layout(T, E, k, d, f).n_counters)
    return fail(MOE_ERR_INVALID_ARG, "spoiled must be -1 or the index of a counter");
  return few(x, logits, nullptr, packed, weights, group, T, d, E, k, f, 1, out, nullptr, nullptr, workspace,
             workspace_bytes, stream, spoiled, static_cast<uint64_t>(limit_ns));
}

moe_status_t moe_selftest_linear_int4_wait(const void* x, int64_t x_stride, const void* packed, int64_t M, int64_t K,
                                           int64_t N, int32_t group, void* out, int64_t out_stride, int32_t row_strips,
                                           int64_t limit_ns, moe_stream_t stream) {
  if (limit_ns < 1 || limit_ns > static_cast<int64_t>(kWaitLimitNs))
    return fail(MOE_ERR_INVALID_ARG, "limit_ns must be in [1, 2e9]");
  if (row_strips < 0) return fail(MOE_ERR_INVALID_ARG, "row_strips must not be negative");
  return linear(x, x_stride, packed, M, K, N, group, out, out_stride, stream, row_strips,
                static_cast<uint64_t>(limit_ns));
}

}  // extern "C"
