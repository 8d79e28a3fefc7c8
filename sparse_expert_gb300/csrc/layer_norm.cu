// Layer norm over the rows of [T, d], forward and backward.
//
//   z  = round(x + residual)  (or x)          mu = mean z
//   r  = 1 / sqrt(mean (z - mu)^2 + eps)      n  = (z - mu) r
//   y  = round(n w + b)
// and for an output gradient dy, g = dy w:
//   dx = r (g - mean g - n mean(g n)) + dz    dw = sum_t dy n    db = sum_t dy
//
// Both directions are bound by memory: every row is read once and written
// once.  A row belongs to a group of `tpr` threads (a power of two), and
// groups walk over the rows.  Three forms, by what the rows allow:
//   - 16-byte chunks (every row, weight and output at a 16-byte boundary, d
//     a whole number of chunks, at most 3 chunks a thread of 512): thread i of
//     a group owns chunks i, i + tpr, ...; it copies its own chunks of the
//     coming rows into its own slots of shared memory asynchronously, several
//     rows ahead, and reads only those slots, so the loads of the next rows
//     cover the reductions of this one without a barrier or a register.
//     Weight, bias and the column sums of the backward stay in registers for
//     all of a thread's rows.
//   - single values (any alignment): thread i owns columns i, i + tpr, ... in
//     registers, so a warp reads neighbouring values.
//   - rows longer than that: sweeps over the row, the later ones out of L2.
// The variance is taken from the deviations from the mean, never as a
// difference of two sums, so a large common offset costs no digits.  Sums
// are fp32 per thread and then trees over lanes and warps, always in the same
// order.
#include <atomic>

#include "common.cuh"
#include "elem.cuh"
#include "internal.h"
#include "launch.cuh"

namespace moe {
namespace {

struct Row {
  const void* ptr;
  int64_t stride;  // elements between rows
};

struct ForwardArgs {
  Row x, res;
  const void* w;
  const void* b;
  bool w_f32;  // weight and bias are fp32, else of the rows' type
  int64_t T;
  int d;
  float eps;
  void* y;
  void* z;
  float* stats;
  int tpr;
};

struct BackwardArgs {
  Row dy, z, dz;
  const float* stats;
  const void* w;
  bool w_f32;
  int64_t T;
  int d;
  void* dx;
  float* partial;  // [blocks][2][d]: the block's sums of dy n, and of dy
  bool want_w, want_b;
  int tpr;
};

constexpr int kMaxWarps = 32;

// Sums over the row's group, in every thread of it.  `red` is one of two
// buffers used in turn: a thread reaches the next sum's barrier only after
// it has read this one's buffer, so one barrier a sum is enough.
__device__ __forceinline__ float2 group_reduce(float2 v, int tpr, float2* red) {
  for (int s = (tpr < 32 ? tpr : 32) >> 1; s > 0; s >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, s);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, s);
  }
  if (tpr <= 32) return v;
  const int lane = threadIdx.x & 31, warps = tpr >> 5, first = threadIdx.x / tpr * warps;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x) / tpr), "r"(tpr) : "memory");
  v = red[first + (lane & (warps - 1))];
  for (int s = warps >> 1; s > 0; s >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, s);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, s);
  }
  return v;
}

__device__ __forceinline__ float group_reduce(float v, int tpr, float2* red) {
  return group_reduce(make_float2(v, 0.0f), tpr, red).x;
}

template <typename T>
__device__ __forceinline__ float param_at(const void* p, bool f32, int j) {
  return f32 ? __ldg(static_cast<const float*>(p) + j) : to_f32(static_cast<const T*>(p)[j]);
}

// A chunk's worth of weight or bias from column j0 (16-byte aligned).
template <typename T>
__device__ __forceinline__ void load_param(const void* p, bool f32, int j0, float* v) {
  if (f32) {
#pragma unroll
    for (int i = 0; i < kChunk<T>; i += 4)
      *reinterpret_cast<float4*>(v + i) = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + j0 + i));
  } else {
    unpack_chunk<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p) + j0)), v);
  }
}

// ---- asynchronous copies of a thread's own chunks
__device__ __forceinline__ void copy_async(uint4* slot, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(slot)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// Rows in flight a thread, by its chunks a row: with three operands at most
// 432 bytes a thread, so 512 threads fill an SM's shared memory.
template <int kChunks>
constexpr int kStages = kChunks == 1 ? 8 : kChunks == 2 ? 4 : 3;
constexpr int kRingThreads = 512;  // resident threads of an SM

template <typename T, int kChunks>
__global__ void __launch_bounds__(kRingThreads) forward_ring_kernel(const ForwardArgs a) {
  constexpr int N = kChunk<T>, S = kStages<kChunks>;
  extern __shared__ uint4 ring[];  // [stage][operand][chunk][thread]
  __shared__ float2 red[2][kMaxWarps];
  const int groups = blockDim.x / a.tpr, lane = threadIdx.x % a.tpr, d = a.d;
  const bool res = a.res.ptr != nullptr;
  const int per_stage = (res ? 2 : 1) * kChunks;
  auto slot = [&](int stage, int operand, int c) {
    return ring + (stage * per_stage + operand * kChunks + c) * blockDim.x + threadIdx.x;
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups;
  const int64_t rounds = (a.T - first + step - 1) / step;
  const int64_t t0 = first + threadIdx.x / a.tpr;
  auto fetch = [&](int64_t round, int stage) {
    const int64_t t = t0 + round * step;
    if (t < a.T) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int j0 = (lane + c * a.tpr) * N;
        if (j0 >= d) continue;
        copy_async(slot(stage, 0, c), static_cast<const T*>(a.x.ptr) + t * a.x.stride + j0);
        if (res) copy_async(slot(stage, 1, c), static_cast<const T*>(a.res.ptr) + t * a.res.stride + j0);
      }
    }
    copy_commit();
  };
  for (int s = 0; s < S - 1; ++s) fetch(s, s);
  float w[kChunks * N], b[kChunks * N];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int j0 = (lane + c * a.tpr) * N;
#pragma unroll
    for (int i = 0; i < N; ++i) w[c * N + i] = 1.0f, b[c * N + i] = 0.0f;
    if (j0 < d && a.w) load_param<T>(a.w, a.w_f32, j0, w + c * N);
    if (j0 < d && a.b) load_param<T>(a.b, a.w_f32, j0, b + c * N);
  }
  const float inv_d = 1.0f / static_cast<float>(d);
  int stage = 0;
  for (int64_t round = 0; round < rounds; ++round) {
    fetch(round + S - 1, stage == 0 ? S - 1 : stage - 1);
    copy_wait<S - 1>();
    const int64_t t = t0 + round * step;
    const bool live = t < a.T;
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int j0 = (lane + c * a.tpr) * N;
      if (j0 >= d || !live) continue;
      float v[N], u[N];
      unpack_chunk<T>(*slot(stage, 0, c), v);
      if (res) {
        // the sum is rounded to the rows' type here: it is what the caller
        // keeps and what the backward normalises again
        unpack_chunk<T>(*slot(stage, 1, c), u);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += u[i];
        const uint4 z = pack_chunk<T>(v);
        *slot(stage, 0, c) = z;
        *reinterpret_cast<uint4*>(static_cast<T*>(a.z) + t * d + j0) = z;
        unpack_chunk<T>(z, v);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) s += v[i];
    }
    const float mu = group_reduce(s, a.tpr, red[0]) * inv_d;
    s = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if ((lane + c * a.tpr) * N >= d || !live) continue;
      float v[N];
      unpack_chunk<T>(*slot(stage, 0, c), v);
#pragma unroll
      for (int i = 0; i < N; ++i) s += (v[i] - mu) * (v[i] - mu);
    }
    const float r = 1.0f / sqrtf(group_reduce(s, a.tpr, red[1]) * inv_d + a.eps);
    if (live && lane == 0) {
      a.stats[t] = mu;
      a.stats[a.T + t] = r;
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int j0 = (lane + c * a.tpr) * N;
      if (j0 >= d || !live) continue;
      float v[N];
      unpack_chunk<T>(*slot(stage, 0, c), v);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = (v[i] - mu) * r * w[c * N + i] + b[c * N + i];
      *reinterpret_cast<uint4*>(static_cast<T*>(a.y) + t * d + j0) = pack_chunk<T>(v);
    }
    stage = stage == S - 1 ? 0 : stage + 1;
  }
}

template <typename T, int kValues>
__global__ void __launch_bounds__(1024) forward_values_kernel(const ForwardArgs a) {
  __shared__ float2 red[2][kMaxWarps];
  const int groups = blockDim.x / a.tpr, lane = threadIdx.x % a.tpr;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / a.tpr;
  const bool live = t < a.T;  // groups beyond the last row follow along without memory accesses
  const int64_t row = live ? t : 0;
  const int d = live ? a.d : 0;
  const T* x = static_cast<const T*>(a.x.ptr) + row * a.x.stride;
  float v[kValues];
#pragma unroll
  for (int i = 0; i < kValues; ++i) {
    const int j = lane + i * a.tpr;
    v[i] = j < d ? to_f32(x[j]) : 0.0f;
  }
  if (a.res.ptr) {
    const T* res = static_cast<const T*>(a.res.ptr) + row * a.res.stride;
    T u[kValues];
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
      const int j = lane + i * a.tpr;
      u[i] = j < d ? res[j] : from_f32<T>(0.0f);
    }
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
      const int j = lane + i * a.tpr;
      const T z = from_f32<T>(v[i] + to_f32(u[i]));
      v[i] = to_f32(z);
      if (j < d) static_cast<T*>(a.z)[row * a.d + j] = z;
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kValues; ++i) s += v[i];
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const float mu = group_reduce(s, a.tpr, red[0]) * inv_d;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < kValues; ++i)
    if (lane + i * a.tpr < d) s += (v[i] - mu) * (v[i] - mu);
  const float r = 1.0f / sqrtf(group_reduce(s, a.tpr, red[1]) * inv_d + a.eps);
  if (live && lane == 0) {
    a.stats[t] = mu;
    a.stats[a.T + t] = r;
  }
#pragma unroll
  for (int i = 0; i < kValues; ++i) {
    const int j = lane + i * a.tpr;
    if (j >= d) continue;
    float y = (v[i] - mu) * r;
    if (a.w) y *= param_at<T>(a.w, a.w_f32, j);
    if (a.b) y += param_at<T>(a.b, a.w_f32, j);
    static_cast<T*>(a.y)[row * a.d + j] = from_f32<T>(y);
  }
}

// One block a row, one value a thread and step.
template <typename T>
__global__ void __launch_bounds__(1024) forward_long_kernel(const ForwardArgs a) {
  __shared__ float2 red[2][kMaxWarps];
  const int64_t t = blockIdx.x;
  const T* x = static_cast<const T*>(a.x.ptr) + t * a.x.stride;
  const T* res = static_cast<const T*>(a.res.ptr) + (a.res.ptr ? t * a.res.stride : 0);
  T* z = static_cast<T*>(a.z) + t * a.d;
  float s = 0.0f;
  for (int j = threadIdx.x; j < a.d; j += blockDim.x) {
    float v = to_f32(x[j]);
    if (a.res.ptr) {
      const T rounded = from_f32<T>(v + to_f32(res[j]));
      z[j] = rounded;
      v = to_f32(rounded);
    }
    s += v;
  }
  // each thread reads back only what it has written itself
  const T* in = a.res.ptr ? z : x;
  const float mu = group_reduce(s, blockDim.x, red[0]) / static_cast<float>(a.d);
  s = 0.0f;
  for (int j = threadIdx.x; j < a.d; j += blockDim.x) {
    const float e = to_f32(in[j]) - mu;
    s += e * e;
  }
  const float r = 1.0f / sqrtf(group_reduce(s, blockDim.x, red[1]) / static_cast<float>(a.d) + a.eps);
  if (threadIdx.x == 0) {
    a.stats[t] = mu;
    a.stats[a.T + t] = r;
  }
  for (int j = threadIdx.x; j < a.d; j += blockDim.x) {
    float v = (to_f32(in[j]) - mu) * r;
    if (a.w) v *= param_at<T>(a.w, a.w_f32, j);
    if (a.b) v += param_at<T>(a.b, a.w_f32, j);
    static_cast<T*>(a.y)[t * a.d + j] = from_f32<T>(v);
  }
}

// The block's column sums from its threads': lanes of a warp that own the
// same columns (tpr below 32) add by a tree, then the warps or groups in
// order through `shared` (slots x d floats).  column(i): value i's column.
template <int kValues, typename Column>
__device__ void write_partial(const BackwardArgs& a, float* sw, float* sb, float* shared, Column column) {
  const int tpr = a.tpr, d = a.d;
  const int slots = tpr < 32 ? blockDim.x >> 5 : blockDim.x / tpr;
  const int slot = tpr < 32 ? threadIdx.x >> 5 : threadIdx.x / tpr;
  const bool owner = tpr >= 32 || (threadIdx.x & 31) < tpr;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (!(which ? a.want_b : a.want_w)) continue;
    float* sum = which ? sb : sw;
    float* out = a.partial + (static_cast<int64_t>(blockIdx.x) * 2 + which) * d;
    if (tpr < 32) {
#pragma unroll
      for (int i = 0; i < kValues; ++i)
        for (int s = 16; s >= tpr; s >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], s);
    }
    if (slots == 1) {
#pragma unroll
      for (int i = 0; i < kValues; ++i)
        if (owner && column(i) < d) out[column(i)] = sum[i];
      continue;
    }
    __syncthreads();  // the ring, or the other sum, is done with `shared`
#pragma unroll
    for (int i = 0; i < kValues; ++i)
      if (owner && column(i) < d) shared[slot * d + column(i)] = sum[i];
    __syncthreads();
    for (int j = threadIdx.x; j < d; j += blockDim.x) {
      float s = shared[j];
      for (int k = 1; k < slots; ++k) s += shared[k * d + j];
      out[j] = s;
    }
  }
}

template <typename T, int kChunks>
__global__ void __launch_bounds__(kRingThreads) backward_ring_kernel(const BackwardArgs a) {
  constexpr int N = kChunk<T>, S = kStages<kChunks>;
  extern __shared__ uint4 ring[];  // [stage][operand][chunk][thread]
  __shared__ float2 red[2][kMaxWarps];
  let_next_start();
  const int groups = blockDim.x / a.tpr, lane = threadIdx.x % a.tpr, d = a.d;
  const bool add = a.dz.ptr != nullptr;
  const int per_stage = (add ? 3 : 2) * kChunks;
  auto slot = [&](int stage, int operand, int c) {
    return ring + (stage * per_stage + operand * kChunks + c) * blockDim.x + threadIdx.x;
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups;
  const int64_t rounds = (a.T - first + step - 1) / step;
  const int64_t t0 = first + threadIdx.x / a.tpr;
  auto fetch = [&](int64_t round, int stage) {
    const int64_t t = t0 + round * step;
    if (t < a.T) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int j0 = (lane + c * a.tpr) * N;
        if (j0 >= d) continue;
        copy_async(slot(stage, 0, c), static_cast<const T*>(a.dy.ptr) + t * a.dy.stride + j0);
        copy_async(slot(stage, 1, c), static_cast<const T*>(a.z.ptr) + t * a.z.stride + j0);
        if (add) copy_async(slot(stage, 2, c), static_cast<const T*>(a.dz.ptr) + t * a.dz.stride + j0);
      }
    }
    copy_commit();
  };
  for (int s = 0; s < S - 1; ++s) fetch(s, s);
  float w[kChunks * N], sw[kChunks * N], sb[kChunks * N];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int j0 = (lane + c * a.tpr) * N;
#pragma unroll
    for (int i = 0; i < N; ++i) w[c * N + i] = 1.0f, sw[c * N + i] = sb[c * N + i] = 0.0f;
    if (j0 < d && a.w) load_param<T>(a.w, a.w_f32, j0, w + c * N);
  }
  const float inv_d = 1.0f / static_cast<float>(d);
  int stage = 0;
  float mu = 0.0f, r = 0.0f;
  if (t0 < a.T) mu = __ldg(a.stats + t0), r = __ldg(a.stats + a.T + t0);
  for (int64_t round = 0; round < rounds; ++round) {
    fetch(round + S - 1, stage == 0 ? S - 1 : stage - 1);
    const int64_t t = t0 + round * step;
    const bool live = t < a.T;
    float next_mu = 0.0f, next_r = 0.0f;
    if (t + step < a.T) next_mu = __ldg(a.stats + t + step), next_r = __ldg(a.stats + a.T + t + step);
    copy_wait<S - 1>();
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if ((lane + c * a.tpr) * N >= d || !live) continue;
      float g[N], n[N];
      unpack_chunk<T>(*slot(stage, 0, c), g);
      unpack_chunk<T>(*slot(stage, 1, c), n);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        n[i] = (n[i] - mu) * r;
        sw[c * N + i] += g[i] * n[i];
        sb[c * N + i] += g[i];
        const float gw = g[i] * w[c * N + i];
        s.x += gw;
        s.y += gw * n[i];
      }
    }
    s = group_reduce(s, a.tpr, red[round & 1]);
    s.x *= inv_d;
    s.y *= inv_d;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int j0 = (lane + c * a.tpr) * N;
      if (j0 >= d || !live) continue;
      float g[N], n[N];
      unpack_chunk<T>(*slot(stage, 0, c), g);
      unpack_chunk<T>(*slot(stage, 1, c), n);
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = (g[i] * w[c * N + i] - s.x - (n[i] - mu) * r * s.y) * r;
      if (add) {
        unpack_chunk<T>(*slot(stage, 2, c), n);
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] += n[i];
      }
      *reinterpret_cast<uint4*>(static_cast<T*>(a.dx) + t * d + j0) = pack_chunk<T>(g);
    }
    mu = next_mu;
    r = next_r;
    stage = stage == S - 1 ? 0 : stage + 1;
  }
  if (a.want_w || a.want_b)
    write_partial<kChunks * N>(a, sw, sb, reinterpret_cast<float*>(ring),
                               [&](int i) { return (lane + i / N * a.tpr) * N + i % N; });
}

template <typename T, int kValues>
__global__ void __launch_bounds__(512) backward_values_kernel(const BackwardArgs a) {
  extern __shared__ uint4 ring[];
  __shared__ float2 red[2][kMaxWarps];
  let_next_start();
  const int groups = blockDim.x / a.tpr, lane = threadIdx.x % a.tpr;
  float sw[kValues], sb[kValues];
#pragma unroll
  for (int i = 0; i < kValues; ++i) sw[i] = sb[i] = 0.0f;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  int parity = 0;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * groups; first < a.T;
       first += static_cast<int64_t>(gridDim.x) * groups, parity ^= 1) {
    const int64_t t = first + threadIdx.x / a.tpr;
    const bool live = t < a.T;
    const int64_t row = live ? t : 0;
    const int d = live ? a.d : 0;
    const T* dy = static_cast<const T*>(a.dy.ptr) + row * a.dy.stride;
    const T* z = static_cast<const T*>(a.z.ptr) + row * a.z.stride;
    const float mu = __ldg(a.stats + row), r = __ldg(a.stats + a.T + row);
    T raw_g[kValues], raw_n[kValues];
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
      const int j = lane + i * a.tpr;
      raw_g[i] = j < d ? dy[j] : from_f32<T>(0.0f);
      raw_n[i] = j < d ? z[j] : from_f32<T>(0.0f);
    }
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
      const int j = lane + i * a.tpr;
      if (j >= d) continue;
      const float g = to_f32(raw_g[i]), n = (to_f32(raw_n[i]) - mu) * r;
      sw[i] += g * n;
      sb[i] += g;
      const float gw = a.w ? g * param_at<T>(a.w, a.w_f32, j) : g;
      s.x += gw;
      s.y += gw * n;
    }
    s = group_reduce(s, a.tpr, red[parity]);
    s.x *= inv_d;
    s.y *= inv_d;
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
      const int j = lane + i * a.tpr;
      if (j >= d) continue;
      const float n = (to_f32(raw_n[i]) - mu) * r;
      const float gw = to_f32(raw_g[i]) * (a.w ? param_at<T>(a.w, a.w_f32, j) : 1.0f);
      float v = (gw - s.x - n * s.y) * r;
      if (a.dz.ptr) v += to_f32(static_cast<const T*>(a.dz.ptr)[row * a.dz.stride + j]);
      static_cast<T*>(a.dx)[row * a.d + j] = from_f32<T>(v);
    }
  }
  if (a.want_w || a.want_b)
    write_partial<kValues>(a, sw, sb, reinterpret_cast<float*>(ring), [&](int i) { return lane + i * a.tpr; });
}

// Rows too long for the registers: dx by a block a row in two sweeps, and
// the column sums by a block for each 256 columns and slice of rows.
template <typename T>
__global__ void __launch_bounds__(1024) backward_long_kernel(const BackwardArgs a) {
  __shared__ float2 red[kMaxWarps];
  const int64_t t = blockIdx.x;
  const T* dy = static_cast<const T*>(a.dy.ptr) + t * a.dy.stride;
  const T* z = static_cast<const T*>(a.z.ptr) + t * a.z.stride;
  const float mu = a.stats[t], r = a.stats[a.T + t];
  float2 s = make_float2(0.0f, 0.0f);
  for (int j = threadIdx.x; j < a.d; j += blockDim.x) {
    const float g = to_f32(dy[j]) * (a.w ? param_at<T>(a.w, a.w_f32, j) : 1.0f);
    s.x += g;
    s.y += g * ((to_f32(z[j]) - mu) * r);
  }
  s = group_reduce(s, blockDim.x, red);
  s.x /= static_cast<float>(a.d);
  s.y /= static_cast<float>(a.d);
  for (int j = threadIdx.x; j < a.d; j += blockDim.x) {
    const float n = (to_f32(z[j]) - mu) * r;
    float v = (to_f32(dy[j]) * (a.w ? param_at<T>(a.w, a.w_f32, j) : 1.0f) - s.x - n * s.y) * r;
    if (a.dz.ptr) v += to_f32(static_cast<const T*>(a.dz.ptr)[t * a.dz.stride + j]);
    static_cast<T*>(a.dx)[t * a.d + j] = from_f32<T>(v);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) column_sums_kernel(const BackwardArgs a, int slices) {
  let_next_start();
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= a.d) return;
  float sw = 0.0f, sb = 0.0f;
  for (int64_t t = blockIdx.y; t < a.T; t += slices) {
    const float g = to_f32(static_cast<const T*>(a.dy.ptr)[t * a.dy.stride + j]);
    const float n = (to_f32(static_cast<const T*>(a.z.ptr)[t * a.z.stride + j]) - __ldg(a.stats + t)) *
                    __ldg(a.stats + a.T + t);
    sw += g * n;
    sb += g;
  }
  float* out = a.partial + static_cast<int64_t>(blockIdx.y) * 2 * a.d;
  if (a.want_w) out[j] = sw;
  if (a.want_b) out[a.d + j] = sb;
}

// dw and db: the blocks' sums added in block order, in 32 interleaved
// partial sums a column.
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
  s = group_sum(part[lane][slice], 32);  // column `slice` of the block
  const int col = blockIdx.x * 32 + slice;
  if (lane == 0 && col < d) out[col] = s;
}

// ---- host
bool rows_on_chunks(const void* p, int64_t stride, int64_t T, int esize) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (T <= 1 || (stride * esize) % 16 == 0);
}

// Threads (a power of two) for a row of `units` chunks or values: up to a
// warp, one each; then as few as hold the row with `most` each.
int threads_per_row(int units, int most) {
  int tpr = 1;
  while (tpr < 32 && tpr < units) tpr *= 2;
  while (tpr * most < units) tpr *= 2;
  return tpr;
}

// Lifts the kernel's shared-memory limit, once for each device.
cudaError_t allow_smem(const void* kernel, std::atomic<uint64_t>& done, size_t bytes) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return err;
}

template <int kChunks>
constexpr size_t ring_bytes(int operands, int block) {
  return static_cast<size_t>(kStages<kChunks>) * operands * kChunks * 16 * block;
}

int grid_of(int64_t T, int groups, int most) {
  const int64_t want = (T + groups - 1) / groups;
  return static_cast<int>(want < most ? want : most);
}

template <typename T, int kChunks>
cudaError_t forward_ring(const ForwardArgs& a, int block, int num_sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t err = allow_smem(reinterpret_cast<const void*>(forward_ring_kernel<T, kChunks>), done,
                                     ring_bytes<kChunks>(2, kRingThreads));
  if (err != cudaSuccess) return err;
  const int grid = grid_of(a.T, block / a.tpr, num_sms * (kRingThreads / block));
  forward_ring_kernel<T, kChunks><<<grid, block, ring_bytes<kChunks>(a.res.ptr ? 2 : 1, block), stream>>>(a);
  return cudaGetLastError();
}

template <typename T, int kValues>
cudaError_t forward_values(const ForwardArgs& a, cudaStream_t stream) {
  const int block = a.tpr < 128 ? 128 : a.tpr, groups = block / a.tpr;
  forward_values_kernel<T, kValues><<<static_cast<unsigned>((a.T + groups - 1) / groups), block, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t forward_typed(ForwardArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int N = kChunk<T>, e = sizeof(T);
  const int wsize = a.w_f32 ? 4 : e;
  const int chunks = (a.d + N - 1) / N;
  const bool on_chunks = a.d % N == 0 && rows_on_chunks(a.x.ptr, a.x.stride, a.T, e) &&
                         (!a.res.ptr || rows_on_chunks(a.res.ptr, a.res.stride, a.T, e)) &&
                         rows_on_chunks(a.y, a.d, a.T, e) && rows_on_chunks(a.z, a.d, a.T, e) &&
                         rows_on_chunks(a.w, 0, 1, wsize) && rows_on_chunks(a.b, 0, 1, wsize);
  if (on_chunks && chunks <= 3 * kRingThreads) {
    a.tpr = threads_per_row(chunks, 3);
    const int block = a.tpr < 256 ? 256 : a.tpr;
    switch ((chunks + a.tpr - 1) / a.tpr) {
      case 1: return forward_ring<T, 1>(a, block, num_sms, stream);
      case 2: return forward_ring<T, 2>(a, block, num_sms, stream);
      default: return forward_ring<T, 3>(a, block, num_sms, stream);
    }
  }
  // at most 8 values a thread: more spill at 1,024 threads
  a.tpr = threads_per_row(a.d, 8);
  if (a.tpr <= 1024)
    return a.d <= a.tpr * 4 ? forward_values<T, 4>(a, stream) : forward_values<T, 8>(a, stream);
  forward_long_kernel<T><<<static_cast<unsigned>(a.T), 1024, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, int kChunks>
cudaError_t backward_ring(const BackwardArgs& a, int block, int num_sms, int* blocks, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t err = allow_smem(reinterpret_cast<const void*>(backward_ring_kernel<T, kChunks>), done,
                                     ring_bytes<kChunks>(3, kRingThreads));
  if (err != cudaSuccess) return err;
  const int most = num_sms * (kRingThreads / block);
  *blocks = grid_of(a.T, block / a.tpr, most < kNormMaxBlocks ? most : kNormMaxBlocks);
  backward_ring_kernel<T, kChunks>
      <<<*blocks, block, ring_bytes<kChunks>(a.dz.ptr ? 3 : 2, block), stream>>>(a);
  return cudaGetLastError();
}

template <typename T, int kValues>
cudaError_t backward_values(const BackwardArgs& a, int num_sms, int* blocks, cudaStream_t stream) {
  const int block = a.tpr < 256 ? 256 : a.tpr, groups = block / a.tpr;
  const int most = num_sms * (kRingThreads / block);
  *blocks = grid_of(a.T, groups, most < kNormMaxBlocks ? most : kNormMaxBlocks);
  const int slots = a.tpr < 32 ? block / 32 : groups;
  const size_t smem = slots > 1 ? static_cast<size_t>(slots) * a.d * 4 : 0;  // at most 8 x 256 floats
  backward_values_kernel<T, kValues><<<*blocks, block, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward_typed(BackwardArgs& a, int num_sms, int* blocks, cudaStream_t stream) {
  constexpr int N = kChunk<T>, e = sizeof(T);
  const int chunks = (a.d + N - 1) / N;
  const bool on_chunks = a.d % N == 0 && rows_on_chunks(a.dy.ptr, a.dy.stride, a.T, e) &&
                         rows_on_chunks(a.z.ptr, a.z.stride, a.T, e) &&
                         (!a.dz.ptr || rows_on_chunks(a.dz.ptr, a.dz.stride, a.T, e)) &&
                         rows_on_chunks(a.dx, a.d, a.T, e) && rows_on_chunks(a.w, 0, 1, a.w_f32 ? 4 : e);
  if (on_chunks && chunks <= 3 * kRingThreads) {
    a.tpr = threads_per_row(chunks, 3);
    const int block = a.tpr < 256 ? 256 : a.tpr;
    switch ((chunks + a.tpr - 1) / a.tpr) {
      case 1: return backward_ring<T, 1>(a, block, num_sms, blocks, stream);
      case 2: return backward_ring<T, 2>(a, block, num_sms, blocks, stream);
      default: return backward_ring<T, 3>(a, block, num_sms, blocks, stream);
    }
  }
  a.tpr = threads_per_row(a.d, a.d <= 2048 ? 8 : 16);
  if (a.tpr <= kRingThreads) {
    const int values = (a.d + a.tpr - 1) / a.tpr;
    if (values <= 4) return backward_values<T, 4>(a, num_sms, blocks, stream);
    if (values <= 8) return backward_values<T, 8>(a, num_sms, blocks, stream);
    return backward_values<T, 16>(a, num_sms, blocks, stream);
  }
  backward_long_kernel<T><<<static_cast<unsigned>(a.T), 1024, 0, stream>>>(a);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || !(a.want_w || a.want_b)) return err;
  *blocks = static_cast<int>(a.T < 64 ? a.T : 64);
  column_sums_kernel<T><<<dim3((a.d + 255) / 256, *blocks), 256, 0, stream>>>(a, *blocks);
  return cudaGetLastError();
}

}  // namespace

size_t norm_backward_workspace_bytes(int64_t T, int d) {
  const int64_t blocks = T < kNormMaxBlocks ? T : kNormMaxBlocks;
  return align_up(static_cast<size_t>(blocks < 1 ? 1 : blocks) * 2 * d * 4);
}

cudaError_t launch_layer_norm(const NormForward& f, int num_sms, cudaStream_t stream) {
  ForwardArgs a{{f.x, f.x_stride}, {f.residual, f.residual_stride}, f.weight, f.bias, f.weight_dtype == MOE_F32,
                f.T, f.d, f.eps, f.y, f.z, f.stats, 0};
  switch (f.dtype) {
    case MOE_F32: return forward_typed<float>(a, num_sms, stream);
    case MOE_BF16: return forward_typed<__nv_bfloat16>(a, num_sms, stream);
    default: return forward_typed<__half>(a, num_sms, stream);
  }
}

cudaError_t launch_layer_norm_backward(const NormBackward& f, int num_sms, cudaStream_t stream) {
  BackwardArgs a{{f.dy, f.dy_stride}, {f.z, f.z_stride}, {f.dz, f.dz_stride}, f.stats, f.weight,
                 f.weight_dtype == MOE_F32, f.T, f.d, f.dx, f.partial, f.dweight != nullptr, f.dbias != nullptr, 0};
  int blocks = 0;
  cudaError_t err;
  switch (f.dtype) {
    case MOE_F32: err = backward_typed<float>(a, num_sms, &blocks, stream); break;
    case MOE_BF16: err = backward_typed<__nv_bfloat16>(a, num_sms, &blocks, stream); break;
    default: err = backward_typed<__half>(a, num_sms, &blocks, stream); break;
  }
  if (err != cudaSuccess || !(a.want_w || a.want_b)) return err;
  return launch_dependent(finish_kernel, dim3((f.d + 31) / 32, 2), 1024, 0, stream, f.partial, blocks, f.d, f.dweight,
                          f.dbias);
}

}  // namespace moe
