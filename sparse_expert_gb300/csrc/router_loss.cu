// The router's auxiliary losses and their gradient in one pass over the
// logits.
//
//   p = softmax(l_t), lse_t = log sum exp l_t, share_e = counts_e / sum,
//   s_t = sum_e p_te share_e
//   balance = E / N sum_t s_t          z = 1 / N sum_t lse_t^2
//   d_te = p_te / N (cb E (share_e - s_t) + 2 cz lse_t)  (+ d_in)
//
// balance needs no column sums: E sum_e share_e mean_t p_te is the mean of
// E s_t, and s_t is what the gradient of the row needs anyway.  So a row is
// read once, its maximum, exponential sum and dot product with the shares
// are reduced inside the lanes that hold it, and its gradient written.
//
// A group of `tpr` lanes (a power of two, up to a warp) holds a row, value
// lane + i * tpr in lane `lane`.
#include "common.cuh"
#include "elem.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

struct Args {
  RouterLoss a;
  int tpr;
};

__device__ __forceinline__ float group_max(float v, int width) {
  for (int s = width >> 1; s > 0; s >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
  return v;
}

// Sum over the block in a fixed order, in thread 0.
__device__ double block_sum(double v, double* red) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double total = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) total += red[i];
  __syncthreads();
  return total;
}

template <int kValues>
__global__ void __launch_bounds__(kThreads) loss_kernel(const Args args) {
  const RouterLoss& a = args.a;
  const int tpr = args.tpr, E = a.E;
  __shared__ double red[kThreads / 32];
  __shared__ double shared_n, shared_counts;
  // N and the total of the counts: every block adds them up for itself
  double kept = 0.0, counted = 0.0;
  if (a.mask)
    for (int64_t t = threadIdx.x; t < a.T; t += kThreads) kept += a.mask[t] != 0 ? 1.0 : 0.0;
  for (int e = threadIdx.x; e < E; e += kThreads) counted += static_cast<double>(a.counts[e]);
  kept = block_sum(kept, red);
  counted = block_sum(counted, red);
  if (threadIdx.x == 0) {
    shared_n = a.mask ? kept : static_cast<double>(a.T);
    shared_counts = counted;
  }
  __syncthreads();
  const float inv_n = shared_n > 0.0 ? static_cast<float>(1.0 / shared_n) : 0.0f;
  const int lane = threadIdx.x % tpr;
  float share[kValues];
#pragma unroll
  for (int i = 0; i < kValues; ++i) {
    const int e = lane + i * tpr;
    share[i] = e < E && shared_counts > 0.0 ? static_cast<float>(a.counts[e] / shared_counts) : 0.0f;
  }
  const float cb = a.balance_coef * static_cast<float>(E), cz = 2.0f * a.z_coef;
  float sum_s = 0.0f, sum_z = 0.0f;
  const int groups = kThreads / tpr;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * groups; t0 < a.T;
       t0 += static_cast<int64_t>(gridDim.x) * groups) {
    const int64_t t = t0 + threadIdx.x / tpr;
    const bool row = t < a.T;
    const bool live = row && (!a.mask || a.mask[t] != 0);
    const int64_t base = t * E;
    float l[kValues];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
      const int e = lane + i * tpr;
      l[i] = live && e < E ? __ldg(a.logits + base + e) : -INFINITY;
      top = fmaxf(top, l[i]);
    }
    top = group_max(top, tpr);
    const bool empty = top == -INFINITY;  // masked, or every logit is -infinity
    float z = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
      // a NaN logit makes z, and so the row's gradient and both losses, NaN
      const float e = empty && l[i] == -INFINITY ? 0.0f : expf(l[i] - top);
      l[i] = e;
      z += e;
      dot += e * share[i];
    }
    z = group_sum(z, tpr);
    dot = group_sum(dot, tpr);
    const float inv_z = empty && z == 0.0f ? 0.0f : 1.0f / z;
    const float s = dot * inv_z;
    const float lse = empty && z == 0.0f ? 0.0f : top + logf(z);
    if (lane == 0) {
      sum_s += s;
      sum_z += lse * lse;
    }
    if (!row) continue;
    const float zl = cz * lse, scale = inv_z * inv_n;
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
      const int e = lane + i * tpr;
      if (e >= E) continue;
      float d = l[i] * scale * (cb * (share[i] - s) + zl);
      if (!live) d = 0.0f;
      if (a.d_in) d += a.d_in[base + e];
      a.d_logits[base + e] = d;
    }
  }
  const double s = block_sum(sum_s, red), z = block_sum(sum_z, red);
  if (threadIdx.x == 0) {
    const double inv = shared_n > 0.0 ? 1.0 / shared_n : 0.0;
    double* out = reinterpret_cast<double*>(a.partial) + 2 * blockIdx.x;
    out[0] = s * E * inv;
    out[1] = z * inv;
  }
}

__global__ void __launch_bounds__(256) finish_kernel(const double* __restrict__ partial, int blocks,
                                                     float* __restrict__ losses) {
  __shared__ double red[8];
  double s = 0.0, z = 0.0;
  for (int b = threadIdx.x; b < blocks; b += 256) {
    s += partial[2 * b];
    z += partial[2 * b + 1];
  }
  s = block_sum(s, red);
  z = block_sum(z, red);
  if (threadIdx.x == 0) {
    losses[0] = static_cast<float>(s);
    losses[1] = static_cast<float>(z);
  }
}

}  // namespace

size_t router_loss_workspace_bytes() { return align_up(kRouterLossMaxBlocks * 2 * sizeof(double)); }

cudaError_t launch_router_loss(const RouterLoss& a, int num_sms, cudaStream_t stream) {
  Args args{a, 1};
  while (args.tpr < 32 && args.tpr * 4 < a.E) args.tpr *= 2;
  const int values = (a.E + args.tpr - 1) / args.tpr;
  const int groups = kThreads / args.tpr;
  const int64_t want = (a.T + groups - 1) / groups;
  const int64_t most = num_sms * 6 < kRouterLossMaxBlocks ? num_sms * 6 : kRouterLossMaxBlocks;
  const int grid = static_cast<int>(want < most ? want : most);
  if (values <= 4) loss_kernel<4><<<grid, kThreads, 0, stream>>>(args);
  else if (values <= 8) loss_kernel<8><<<grid, kThreads, 0, stream>>>(args);
  else if (values <= 12) loss_kernel<12><<<grid, kThreads, 0, stream>>>(args);
  else if (values <= 16) loss_kernel<16><<<grid, kThreads, 0, stream>>>(args);
  else loss_kernel<32><<<grid, kThreads, 0, stream>>>(args);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  finish_kernel<<<1, 256, 0, stream>>>(reinterpret_cast<const double*>(a.partial), grid, a.losses);
  return cudaGetLastError();
}

}  // namespace moe
