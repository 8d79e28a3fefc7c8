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
// accesses, else single values.  Groups walk over the rows; a lane copies its
// own values of the next row into its own slots of shared memory while it
// works on this one, so no barrier is needed and the loads never pause.
//
// The mask is counted by a kernel of its own first: every block needs N, and
// each counting for itself (in the first version) cost more than the losses
// (65,536 tokens: 349 us in all).  A small problem is one cluster of blocks
// that count, and add up the losses, among themselves: one launch.
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
  double* partial;      // [blocks][2], unless one cluster adds up the losses
  int tpr;
  int cluster;          // its blocks, or 0
};

__device__ __forceinline__ float group_max(float v, int width) {
  if (width == 32) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
  } else {
    for (int s = width >> 1; s > 0; s >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
  }
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

// A lane's slots: 16 bytes a vector, or 4 a value, kThreads lanes apart.
template <bool kVec>
constexpr uint32_t kPitch = kThreads * (kVec ? 16 : 4);

template <int kValues, bool kVec, bool kFull>
__device__ __forceinline__ void fetch_row(uint32_t slot, const float* row, int E, int lane, int tpr) {
#pragma unroll
  for (int i = 0; i < kValues; i += kVec ? 4 : 1) {
    const int e = column<kVec>(i, lane, tpr);
    if (!kFull && e >= E) continue;
    if (kVec)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + i / 4 * kPitch<kVec>), "l"(row + e)
                   : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(slot + i * kPitch<kVec>), "l"(row + e) : "memory");
  }
}

template <int kValues, bool kVec, bool kFull>
__device__ __forceinline__ void take_row(uint32_t slot, bool live, float fill, int E, int lane, int tpr,
                                         float2 (&v)[kValues / 2]) {
#pragma unroll
  for (int i = 0; i < kValues; i += kVec ? 4 : 2) {
    const int e = column<kVec>(i, lane, tpr);
    if (kVec) {
      float4 q = make_float4(fill, fill, fill, fill);
      if (live && (kFull || e < E))
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(q.x), "=f"(q.y), "=f"(q.z), "=f"(q.w)
                     : "r"(slot + i / 4 * kPitch<kVec>));
      v[i / 2] = make_float2(q.x, q.y);
      v[i / 2 + (kVec ? 1 : 0)] = kVec ? make_float2(q.z, q.w) : v[i / 2];
    } else {
      v[i / 2] = both(fill);
      if (live && e < E) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[i / 2].x) : "r"(slot + i * kPitch<kVec>));
      if (live && e + tpr < E)
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[i / 2].y) : "r"(slot + (i + 1) * kPitch<kVec>));
    }
  }
}

// 2^v for -126 <= v (0 below).
__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Rows in flight: this one and the next two where a lane has up to 12 values
// (3 resident blocks of 74 KB), else the next one.
template <int kValues>
constexpr int kStages = kValues <= 12 ? 3 : 2;

template <int kValues, bool kVec, bool kFull>
__global__ void __launch_bounds__(kThreads, kValues <= 12 ? 3 : 2) loss_kernel(const Args args) {
  const RouterLoss& a = args.a;
  constexpr int kPairsRow = kValues / 2, S = kStages<kValues>;
  constexpr uint32_t kOperand = kValues / (kVec ? 4 : 1) * kPitch<kVec>;
  const int tpr = args.tpr, E = a.E;
  extern __shared__ uint4 ring[];  // [stage][operand][vector or value][thread]
  __shared__ int64_t red_i[kThreads / 32];
  __shared__ double red[kThreads / 32], block_losses[2];
  let_next_start();
  const int lane = threadIdx.x % tpr;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / tpr);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads / tpr);
  const int64_t rounds = (a.T - first + step - 1) / step;
  int64_t t = first + threadIdx.x / tpr;
  auto kept_row = [&](int64_t row) { return row < a.T && (!a.mask || __ldg(a.mask + row) != 0); };
  // a masked row of a gradient accumulated in place is left as it is
  const bool in_place = a.d_in && a.d_in == a.d_logits;
  const uint32_t own = smem_addr(ring) + threadIdx.x * (kVec ? 16 : 4), stage_bytes = (a.d_in ? 2 : 1) * kOperand;
  int64_t ahead = t;
  bool ahead_live = kept_row(ahead);
  uint32_t live_bits = 0;  // bit k: the row k rounds after this one is kept
  auto fetch = [&](uint32_t stage, int round) {
    if (ahead_live) fetch_row<kValues, kVec, kFull>(stage, a.logits + ahead * E, E, lane, tpr);
    if (a.d_in && ahead < a.T && (ahead_live || !in_place))
      fetch_row<kValues, kVec, kFull>(stage + kOperand, a.d_in + ahead * E, E, lane, tpr);
    asm volatile("cp.async.commit_group;" ::: "memory");
    live_bits |= static_cast<uint32_t>(ahead_live) << round;
    ahead += step;
    ahead_live = kept_row(ahead);
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(own + s * stage_bytes, s);
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
  } else if (a.mask) {
    int64_t part = 0;
    for (int64_t i = threadIdx.x; i < a.T; i += kThreads) part += a.mask[i] != 0;
    n = block_sum(part, red_i);
  }
  const float inv_n = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
  const float cb = a.balance_coef * static_cast<float>(E), cz = 2.0f * a.z_coef;
  constexpr float kLog2e = 1.4426950408889634f;
  float sum_s = 0.0f, sum_z = 0.0f;
  uint32_t stage = own, next = own + (S - 1) * stage_bytes;
  for (int64_t round = 0; round < rounds; ++round, t += step, live_bits >>= 1) {
    fetch(next, S - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    const bool row = t < a.T, live = live_bits & 1u, write = row && (live || !in_place);
    float2 l[kPairsRow], before[kPairsRow];
    take_row<kValues, kVec, kFull>(stage, live, -INFINITY, E, lane, tpr, l);
    if (a.d_in) take_row<kValues, kVec, kFull>(stage + kOperand, write, 0.0f, E, lane, tpr, before);
    next = stage;
    stage = stage + stage_bytes == own + S * stage_bytes ? own : stage + stage_bytes;
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
      // e^x as the square of 2^(x log2(e) / 2), which stays above the
      // denormals down to the smallest of them
      const float2 e = mul2(add2(l[i], shift), both(0.5f * kLog2e));
      l[i] = make_float2(exp2_approx(e.x), exp2_approx(e.y));
      l[i] = mul2(l[i], l[i]);
      z2 = add2(z2, l[i]);
      dot2 = fma2(l[i], share[i], dot2);
    }
    const float z = group_sum(z2.x + z2.y, tpr), dot = group_sum(dot2.x + dot2.y, tpr);
    const bool empty = z == 0.0f;
    const float inv_z = empty ? 0.0f : __fdividef(1.0f, z);  // z in [1, E]
    const float s = dot * inv_z;
    const float lse = empty ? 0.0f : top + __logf(z);
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
        if (kFull || e < E) *reinterpret_cast<float4*>(out + e) = make_float4(lo.x, lo.y, hi.x, hi.y);
      } else {
        if (e < E) out[e] = lo.x;
        if (e + tpr < E) out[e + tpr] = lo.y;
      }
    }
  }
  // every lane of a group carries the row's sums: one of them counts
  const double s = block_sum(lane == 0 ? static_cast<double>(sum_s) : 0.0, red);
  const double z = block_sum(lane == 0 ? static_cast<double>(sum_z) : 0.0, red);
  const double inv = n > 0 ? 1.0 / static_cast<double>(n) : 0.0;
  if (!args.cluster) {
    if (threadIdx.x == 0) {
      args.partial[2 * blockIdx.x] = s * E * inv;
      args.partial[2 * blockIdx.x + 1] = z * inv;
    }
    return;
  }
  if (threadIdx.x == 0) {
    block_losses[0] = s * E * inv;
    block_losses[1] = z * inv;
  }
  cluster_sync();
  if (cluster_rank() == 0 && threadIdx.x < 2) {
    double sum = 0.0;
    for (int k = 0; k < args.cluster; ++k) sum += remote_f64(block_losses + threadIdx.x, k);
    a.losses[threadIdx.x] = static_cast<float>(sum);
  }
  cluster_sync();  // no block leaves while another reads its sums
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
template <int kValues, bool kVec, bool kFull>
cudaError_t launch_one(const Args& args, int grid, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr size_t operand = kStages<kValues> * (kValues / (kVec ? 4 : 1)) * static_cast<size_t>(kPitch<kVec>);
  const cudaError_t err = allow(reinterpret_cast<const void*>(loss_kernel<kValues, kVec, kFull>), done, 2 * operand, true);
  if (err != cudaSuccess) return err;
  const size_t smem = (args.a.d_in ? 2 : 1) * operand;
  if (args.cluster) return launch_cluster(loss_kernel<kValues, kVec, kFull>, args.cluster, kThreads, smem, stream, args);
  if (args.kept) return launch_dependent(loss_kernel<kValues, kVec, kFull>, grid, kThreads, smem, stream, args);
  loss_kernel<kValues, kVec, kFull><<<grid, kThreads, smem, stream>>>(args);
  return cudaGetLastError();
}

template <bool kVec, bool kFull>
cudaError_t launch_losses(const Args& args, int values, int grid, cudaStream_t stream) {
  if (values <= 4) return launch_one<4, kVec, kFull>(args, grid, stream);
  if (values <= 8) return launch_one<8, kVec, kFull>(args, grid, stream);
  if (values <= 12) return launch_one<12, kVec, kFull>(args, grid, stream);
  if (values <= 16) return launch_one<16, kVec, kFull>(args, grid, stream);
  return launch_one<32, kVec, kFull>(args, grid, stream);
}

// A row fills all of its lanes' values where E is so many: nothing to check.
cudaError_t launch_losses(const Args& args, bool vec, int values, int grid, cudaStream_t stream) {
  if (!vec) return launch_losses<false, false>(args, values, grid, stream);
  const bool full = args.a.E == args.tpr * values && (values <= 16 || values == 32);
  return full ? launch_losses<true, true>(args, values, grid, stream)
              : launch_losses<true, false>(args, values, grid, stream);
}

constexpr size_t kPartialBytes = kRouterLossMaxBlocks * 2 * sizeof(double);

}  // namespace

size_t router_loss_workspace_bytes() { return align_up(kPartialBytes + kCountBlocks * sizeof(int32_t)); }

cudaError_t launch_router_loss(const RouterLoss& a, int num_sms, cudaStream_t stream) {
  auto* kept = reinterpret_cast<int32_t*>(static_cast<char*>(a.workspace) + kPartialBytes);
  Args args{a, nullptr, static_cast<double*>(a.workspace), 1, 0};
  const uintptr_t low = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.d_in) |
                        reinterpret_cast<uintptr_t>(a.d_logits);
  const bool vec = a.E % 4 == 0 && low % 16 == 0;
  const int units = vec ? a.E / 4 : a.E, per = vec ? 1 : 4;
  while (args.tpr < 32 && args.tpr * per < units) args.tpr *= 2;
  const int values = (units + args.tpr - 1) / args.tpr * (vec ? 4 : 1);
  const int groups = kThreads / args.tpr;
  const int64_t want = (a.T + groups - 1) / groups;
  cudaError_t err;
  // one cluster up to 2 rounds of the largest: further rounds cost more than
  // the other launches
  if (want <= kClusterMost * 2) {
    args.cluster = 1;
    while (args.cluster < want && args.cluster < kClusterMost) args.cluster *= 2;
    return launch_losses(args, vec, values, 0, stream);
  }
  const int64_t most = num_sms * (values <= 12 ? 3 : 2);
  const int grid = static_cast<int>(want < most ? want : most);
  if (a.mask) {
    args.kept = kept;
    count_kernel<<<kCountBlocks, kThreads, 0, stream>>>(a.mask, a.T, kept);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
  }
  err = launch_losses(args, vec, values, grid, stream);
  if (err != cudaSuccess) return err;
  return launch_dependent(finish_kernel, 1, kThreads, 0, stream, args.partial, grid, a.losses);
}

}  // namespace moe
