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
// A group of `tpr` lanes (a power of two, up to a warp) holds a row: vectors
// of four values lane, lane + tpr, ... where rows and E allow 16-byte
// accesses, else single values.  Enough warps are resident to cover a row's
// loads by the others' arithmetic, which runs on pairs of values.
//
// The mask is counted by a kernel of its own first: every block needs N, and
// each counting for itself (in the first version) cost more than the losses
// (65,536 tokens: 349 us in all).
#include "common.cuh"
#include "elem.cuh"
#include "internal.h"
#include "launch.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kCountBlocks = 64;

struct Args {
  RouterLoss a;
  const int32_t* kept;  // [kCountBlocks] tokens kept, by the counting kernel; null without a mask
  double* partial;      // [blocks][2]
  int tpr;
};

__device__ __forceinline__ float group_max(float v, int width) {
  for (int s = width >> 1; s > 0; s >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
  return v;
}

// Sum over the block in a fixed order, in every thread.
template <typename T>
__device__ T block_sum(T v, T* red) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  T total = 0;
  for (int i = 0; i < kThreads / 32; ++i) total += red[i];
  __syncthreads();
  return total;
}

__global__ void __launch_bounds__(kThreads) count_kernel(const uint8_t* __restrict__ mask, int64_t T,
                                                         int32_t* __restrict__ kept) {
  __shared__ int red[kThreads / 32];
  let_next_start();
  int n = 0;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  // bytes up to a 16-byte boundary, whole vectors, the rest
  int64_t head = static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(mask) & 15)) & 15);
  if (head > T) head = T;
  const int64_t vectors = (T - head) / 16;
  for (int64_t i = first; i < vectors; i += stride) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(mask + head) + i);
    // a byte of __vcmpgtu4 is 255 where the mask's byte is above 0
    n += (__popc(__vcmpgtu4(u.x, 0)) + __popc(__vcmpgtu4(u.y, 0)) + __popc(__vcmpgtu4(u.z, 0)) +
          __popc(__vcmpgtu4(u.w, 0))) >> 3;
  }
  const int64_t tail = head + vectors * 16;
  if (first < head) n += mask[first] != 0;
  if (tail + first < T) n += mask[tail + first] != 0;
  n = block_sum(n, red);
  if (threadIdx.x == 0) kept[blockIdx.x] = n;
}

// Column of value i of a lane.
template <bool kVec>
__device__ __forceinline__ int column(int i, int lane, int tpr) {
  return kVec ? ((i >> 2) * tpr + lane) * 4 + (i & 3) : i * tpr + lane;
}

template <int kValues, bool kVec>
__device__ __forceinline__ void load_row(const float* row, bool live, float fill, int E, int lane, int tpr,
                                         float2 (&v)[kValues / 2]) {
#pragma unroll
  for (int i = 0; i < kValues; i += kVec ? 4 : 2) {
    const int e = column<kVec>(i, lane, tpr);
    if (kVec) {
      float4 q = make_float4(fill, fill, fill, fill);
      if (live && e < E) q = *reinterpret_cast<const float4*>(row + e);
      v[i / 2] = make_float2(q.x, q.y);
      v[i / 2 + 1] = make_float2(q.z, q.w);
    } else {
      v[i / 2].x = live && e < E ? row[e] : fill;
      v[i / 2].y = live && e + tpr < E ? row[e + tpr] : fill;
    }
  }
}

__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

template <int kValues, bool kVec>
__global__ void __launch_bounds__(kThreads, kValues <= 12 ? 4 : 2) loss_kernel(const Args args) {
  const RouterLoss& a = args.a;
  constexpr int kPairsRow = kValues / 2;
  const int tpr = args.tpr, E = a.E;
  __shared__ int64_t red_i[kThreads / 32];
  __shared__ double red[kThreads / 32];
  let_next_start();
  const int lane = threadIdx.x % tpr;
  int64_t counted = 0;
  for (int e = threadIdx.x; e < E; e += kThreads) counted += a.counts[e];
  counted = block_sum(counted, red_i);
  // fp32 quotients: counts and their total are exact to 24 bits
  const float total = static_cast<float>(counted);
  float2 share[kPairsRow];
#pragma unroll
  for (int i = 0; i < kValues; ++i) {
    const int e = column<kVec>(i, lane, tpr);
    const float q = e < E && counted > 0 ? static_cast<float>(a.counts[e]) / total : 0.0f;
    if (i & 1) share[i / 2].y = q;
    else share[i / 2].x = q;
  }
  int64_t n = a.T;
  if (args.kept) {
    wait_for_previous();
    int64_t part = threadIdx.x < kCountBlocks ? args.kept[threadIdx.x] : 0;
    n = block_sum(part, red_i);
  }
  const float inv_n = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
  const float cb = a.balance_coef * static_cast<float>(E), cz = 2.0f * a.z_coef;
  constexpr float kLog2e = 1.4426950408889634f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / tpr);
  float sum_s = 0.0f, sum_z = 0.0f;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads / tpr); first < a.T; first += step) {
    const int64_t t = first + threadIdx.x / tpr;
    const bool row = t < a.T;
    const bool live = row && (!a.mask || a.mask[t] != 0);
    // a masked row of a gradient accumulated in place is left as it is
    const bool write = row && (live || !a.d_in || a.d_in != a.d_logits);
    float2 l[kPairsRow], before[kPairsRow];
    load_row<kValues, kVec>(a.logits + t * E, live, -INFINITY, E, lane, tpr, l);
    if (a.d_in) load_row<kValues, kVec>(a.d_in + t * E, write, 0.0f, E, lane, tpr, before);
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPairsRow; ++i) top = fmaxf(top, fmaxf(l[i].x, l[i].y));
    top = group_max(top, tpr);
    // a row without a finite or infinite logit above -infinity (masked, or
    // every expert taken out) is shifted by 0: its exponentials are zero.  A
    // NaN makes z, and so the row's gradient and both losses, NaN
    const float2 shift = both(top == -INFINITY ? 0.0f : -top);
    float2 z2 = both(0.0f), dot2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < kPairsRow; ++i) {
      const float2 e = mul2(add2(l[i], shift), both(kLog2e));
      l[i] = make_float2(exp2_approx(e.x), exp2_approx(e.y));
      z2 = add2(z2, l[i]);
      dot2 = fma2(l[i], share[i], dot2);
    }
    const float z = group_sum(z2.x + z2.y, tpr), dot = group_sum(dot2.x + dot2.y, tpr);
    const bool empty = z == 0.0f;
    const float inv_z = empty ? 0.0f : 1.0f / z;
    const float s = dot * inv_z;
    const float lse = empty ? 0.0f : top + logf(z);
    sum_s += s;
    sum_z += lse * lse;
    if (!write) continue;
    // p / N (cb (share - s) + cz lse) = e (scale_b share + scale_0)
    const float scale = inv_z * inv_n;
    const float2 scale_b = both(scale * cb), scale_0 = both(scale * (cz * lse - cb * s));
    float* out = a.d_logits + t * E;
#pragma unroll
    for (int i = 0; i < kPairsRow; ++i) {
      l[i] = mul2(l[i], fma2(scale_b, share[i], scale_0));
      if (a.d_in) l[i] = add2(l[i], before[i]);
    }
#pragma unroll
    for (int i = 0; i < kValues; i += kVec ? 4 : 2) {
      const int e = column<kVec>(i, lane, tpr);
      const float2 lo = l[i / 2];
      if (kVec) {
        const float2 hi = l[i / 2 + (kVec ? 1 : 0)];
        if (e < E) *reinterpret_cast<float4*>(out + e) = make_float4(lo.x, lo.y, hi.x, hi.y);
      } else {
        if (e < E) out[e] = lo.x;
        if (e + tpr < E) out[e + tpr] = lo.y;
      }
    }
  }
  // every lane of a group carries the row's sums: one of them counts
  const double s = block_sum(lane == 0 ? static_cast<double>(sum_s) : 0.0, red);
  const double z = block_sum(lane == 0 ? static_cast<double>(sum_z) : 0.0, red);
  if (threadIdx.x == 0) {
    const double inv = n > 0 ? 1.0 / static_cast<double>(n) : 0.0;
    args.partial[2 * blockIdx.x] = s * E * inv;
    args.partial[2 * blockIdx.x + 1] = z * inv;
  }
}

__global__ void __launch_bounds__(kThreads) finish_kernel(const double* __restrict__ partial, int blocks,
                                                          float* __restrict__ losses) {
  __shared__ double red[kThreads / 32];
  wait_for_previous();
  double s = 0.0, z = 0.0;
  for (int b = threadIdx.x; b < blocks; b += kThreads) {
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

// After the counting kernel the losses may start early (they wait for its
// result); without it they follow the caller's work as any launch does.
template <int kValues, bool kVec>
cudaError_t launch_one(const Args& args, int grid, cudaStream_t stream) {
  if (args.kept) return launch_dependent(loss_kernel<kValues, kVec>, grid, kThreads, 0, stream, args);
  loss_kernel<kValues, kVec><<<grid, kThreads, 0, stream>>>(args);
  return cudaGetLastError();
}

template <bool kVec>
cudaError_t launch_losses(const Args& args, int values, int grid, cudaStream_t stream) {
  if (values <= 4) return launch_one<4, kVec>(args, grid, stream);
  if (values <= 8) return launch_one<8, kVec>(args, grid, stream);
  if (values <= 12) return launch_one<12, kVec>(args, grid, stream);
  if (values <= 16) return launch_one<16, kVec>(args, grid, stream);
  return launch_one<32, kVec>(args, grid, stream);
}

constexpr size_t kPartialBytes = kRouterLossMaxBlocks * 2 * sizeof(double);

}  // namespace

size_t router_loss_workspace_bytes() { return align_up(kPartialBytes + kCountBlocks * sizeof(int32_t)); }

cudaError_t launch_router_loss(const RouterLoss& a, int num_sms, cudaStream_t stream) {
  auto* kept = reinterpret_cast<int32_t*>(static_cast<char*>(a.workspace) + kPartialBytes);
  Args args{a, a.mask ? kept : nullptr, static_cast<double*>(a.workspace), 1};
  const uintptr_t low = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.d_in) |
                        reinterpret_cast<uintptr_t>(a.d_logits);
  const bool vec = a.E % 4 == 0 && low % 16 == 0;
  const int units = vec ? a.E / 4 : a.E, per = vec ? 1 : 4;
  while (args.tpr < 32 && args.tpr * per < units) args.tpr *= 2;
  const int values = (units + args.tpr - 1) / args.tpr * (vec ? 4 : 1);
  const int groups = kThreads / args.tpr;
  const int64_t want = (a.T + groups - 1) / groups;
  const int64_t most = num_sms * 4 < kRouterLossMaxBlocks ? num_sms * 4 : kRouterLossMaxBlocks;
  const int grid = static_cast<int>(want < most ? want : most);
  cudaError_t err;
  if (a.mask) {
    count_kernel<<<kCountBlocks, kThreads, 0, stream>>>(a.mask, a.T, kept);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
  }
  err = vec ? launch_losses<true>(args, values, grid, stream) : launch_losses<false>(args, values, grid, stream);
  if (err != cudaSuccess) return err;
  return launch_dependent(finish_kernel, 1, kThreads, 0, stream, args.partial, grid, a.losses);
}

}  // namespace moe
