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
//   - rings of 16-byte chunks, where all operands of a row lie alike within
//     16 bytes (contiguous tensors of any d do) and 3 chunks a thread of 512
//     hold a row: thread i of a group owns the aligned chunks i, i + tpr, ...
//     of its rows; it copies its own chunks of the coming rows into its own
//     slots of shared memory asynchronously, several rows ahead, and reads
//     only those slots, so the loads of the next rows cover the reductions of
//     this one without a barrier or a register.  Weight, bias and the column
//     sums of the backward stay in registers for all of a thread's rows.
//     Rows that do not start on a chunk: a group steps over rows in multiples
//     of a chunk's values, after which a row starts at the same place within
//     16 bytes, so a thread's columns stay the same; only the first and the
//     last chunk of such a row are partial, and their other values masked.
//   - single values (operands that lie differently): thread i owns columns
//     i, i + tpr, ... in registers, so a warp reads neighbouring values.
//   - rows longer than that: sweeps over the row, the later ones out of L2.
// The variance is taken from the deviations from the mean, never as a
// difference of two sums, so a large common offset costs no digits.  Sums
// are fp32 per thread and then trees over lanes and warps, always in the same
// order.
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
  float* dw;  // the sums over all blocks, where one cluster holds them
  float* db;
  bool want_w, want_b;
  int tpr;
  int cluster;  // blocks of that cluster, or 0: the sums go to `partial`
};

constexpr int kMaxWarps = 32;

__device__ __forceinline__ float shuffle_add(float v, int s) { return v + __shfl_xor_sync(0xffffffffu, v, s); }
__device__ __forceinline__ float2 shuffle_add(float2 v, int s) {
  return make_float2(shuffle_add(v.x, s), shuffle_add(v.y, s));
}

// Sum over the lanes of a warp that belong to the row: all of them, or the
// aligned group of tpr.
template <typename V>
__device__ __forceinline__ V warp_reduce(V v, int tpr) {
  if (tpr >= 32) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v = shuffle_add(v, s);
  } else {
    for (int s = tpr >> 1; s > 0; s >>= 1) v = shuffle_add(v, s);
  }
  return v;
}

// Tree over the group's warps, whose values lie in lanes modulo `warps`.
template <typename V>
__device__ __forceinline__ V over_warps(V v, int warps) {
#pragma unroll
  for (int s = kMaxWarps / 2; s > 0; s >>= 1)
    if (s < warps) v = shuffle_add(v, s);
  return v;
}

// Hands each warp's value to the whole group: the calling lane gets that of
// warp lane mod warps.  `red` is one of two buffers used in turn: a thread
// reaches the next exchange's barrier only after it has read this one's
// buffer, so one barrier each is enough.
__device__ __forceinline__ float2 exchange(float2 v, int tpr, float2* red) {
  const int lane = threadIdx.x & 31, warps = tpr >> 5, group = threadIdx.x / tpr;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
  return red[group * warps + (lane & (warps - 1))];
}

// Sums over the row's group, in every thread of it.
__device__ __forceinline__ float2 group_reduce(float2 v, int tpr, float2* red) {
  v = warp_reduce(v, tpr);
  return tpr <= 32 ? v : over_warps(exchange(v, tpr, red), tpr >> 5);
}

__device__ __forceinline__ float group_reduce(float v, int tpr, float2* red) {
  v = warp_reduce(v, tpr);
  return tpr <= 32 ? v : over_warps(exchange(make_float2(v, 0.0f), tpr, red).x, tpr >> 5);
}

template <typename T>
__device__ __forceinline__ float param_at(const void* p, bool f32, int j) {
  return f32 ? __ldg(static_cast<const float*>(p) + j) : to_f32(static_cast<const T*>(p)[j]);
}

// ---- asynchronous copies of a thread's own chunks
__device__ __forceinline__ void copy_async(uint32_t slot, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot), "l"(src) : "memory");
}
// The first `bytes` of the chunk, the rest zero.
__device__ __forceinline__ void copy_async_part(uint32_t slot, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ uint4 load_slot(uint32_t slot) {
  uint4 u;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(slot));
  return u;
}
// One block of 512 threads an SM.  Rows in flight, by a thread's chunks a
// row: what the SM's shared memory holds with two operands (forward) or
// three (backward): at most 432 bytes a thread.
constexpr int kRingThreads = 512;
constexpr uint32_t kPitch = kRingThreads * 16;  // bytes between a thread's slots
template <int kChunks>
constexpr int kForwardStages = kChunks == 1 ? 8 : kChunks == 2 ? 6 : 4;
template <int kChunks>
constexpr int kBackwardStages = kChunks == 1 ? 8 : kChunks == 2 ? 4 : 3;

// Where a thread's chunks lie, for all of its rows.
template <typename T, int kChunks, bool kAligned>
struct Place {
  static constexpr int N = kChunk<T>;
  int j0[kChunks];  // first column of each chunk: from -off up, at least d for a chunk beyond the row
  int d;
  __device__ __forceinline__ Place(int lane, int tpr, int d_, int off) : d(d_) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) j0[c] = (lane + c * tpr) * N - (kAligned ? 0 : off);
  }
  __device__ __forceinline__ bool any(int c) const { return j0[c] < d; }
  __device__ __forceinline__ bool whole(int c) const { return kAligned || (j0[c] >= 0 && j0[c] + N <= d); }
  // Copies the chunk.  A partial first chunk is copied whole: its 16 aligned
  // bytes hold at least one value of the row, so they lie inside the
  // row's allocation.  A last chunk ends with the row.
  __device__ __forceinline__ void fetch(uint32_t slot, const T* row, int c) const {
    if (kAligned || j0[c] + N <= d) copy_async(slot, row + j0[c]);
    else copy_async_part(slot, row + j0[c], (d - j0[c]) * static_cast<int>(sizeof(T)));
  }
  // Values outside the row become `fill`.
  __device__ __forceinline__ void mask(int c, float2* v, float fill) const {
    if (whole(c)) return;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const int j = j0[c] + 2 * i;
      if (j < 0 || j >= d) v[i].x = fill;
      if (j + 1 < 0 || j + 1 >= d) v[i].y = fill;
    }
  }
  __device__ __forceinline__ void store(T* row, int c, const uint4& u) const {
    if (whole(c)) {
      *reinterpret_cast<uint4*>(row + j0[c]) = u;
      return;
    }
    float v[N];
    unpack_chunk<T>(u, v);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (j0[c] + i >= 0 && j0[c] + i < d) row[j0[c] + i] = from_f32<T>(v[i]);
  }
  // The chunk's weights or biases.
  __device__ __forceinline__ void params(int c, const void* p, bool f32, float missing, float2* v) const {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) v[i] = both(missing);
    if (!p || !any(c)) return;
    if (kAligned) {
      if (f32) {
#pragma unroll
        for (int i = 0; i < N / 2; i += 2) {
          const float4 q = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + j0[c] + 2 * i));
          v[i] = make_float2(q.x, q.y);
          v[i + 1] = make_float2(q.z, q.w);
        }
      } else {
        unpack_pairs<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p) + j0[c])), v);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const int j = j0[c] + 2 * i;
      if (j >= 0 && j < d) v[i].x = param_at<T>(p, f32, j);
      if (j + 1 >= 0 && j + 1 < d) v[i].y = param_at<T>(p, f32, j + 1);
    }
  }
};

template <typename T>
__device__ __forceinline__ int row_offset(const Row& rows, int64_t t) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(static_cast<const T*>(rows.ptr) + t * rows.stride) & 15) /
                          sizeof(T));
}

template <typename T, int kChunks, bool kAligned>
__global__ void __launch_bounds__(kRingThreads, 1) forward_ring_kernel(const ForwardArgs a) {
  constexpr int P = kPairs<T>, S = kForwardStages<kChunks>;
  extern __shared__ uint4 ring[];  // [stage][operand][chunk][thread]
  __shared__ float2 red[2][kMaxWarps];
  const int groups = kRingThreads / a.tpr, lane = threadIdx.x % a.tpr;
  const bool res = a.res.ptr != nullptr;
  const uint32_t own = smem_addr(ring) + threadIdx.x * 16, stage_bytes = (res ? 2 : 1) * kChunks * kPitch;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups;
  const int64_t rounds = (a.T - first + step - 1) / step;
  int64_t t = first + threadIdx.x / a.tpr;
  const Place<T, kChunks, kAligned> at(lane, a.tpr, a.d, kAligned ? 0 : row_offset<T>(a.x, t));
  const T* x = static_cast<const T*>(a.x.ptr) + t * a.x.stride;
  const T* r_row = static_cast<const T*>(a.res.ptr) + (res ? t * a.res.stride : 0);
  int64_t ahead = t;  // the row that x and r_row stand at
  auto fetch = [&](uint32_t stage) {
    if (ahead < a.T) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (!at.any(c)) continue;
        at.fetch(stage + c * kPitch, x, c);
        if (res) at.fetch(stage + (kChunks + c) * kPitch, r_row, c);
      }
    }
    copy_commit();
    ahead += step;
    x += step * a.x.stride;
    if (res) r_row += step * a.res.stride;
  };
  for (int s = 0; s < S - 1; ++s) fetch(own + s * stage_bytes);
  float2 w[kChunks * P], b[kChunks * P];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    at.params(c, a.w, a.w_f32, 1.0f, w + c * P);
    at.params(c, a.b, a.w_f32, 0.0f, b + c * P);
  }
  const float inv_d = 1.0f / static_cast<float>(a.d);
  // Mean and variance take one exchange: a warp (or a group inside one) takes
  // the deviations from its own mean, and the warps' sums q_i of their n_i
  // values about their means m_i join as q = sum q_i + n_i (m_i - mu)^2.
  int count = 0;
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
    if (at.any(c)) count += min(at.j0[c] + 2 * P, a.d) - max(at.j0[c], 0);
  const float n_warp = warp_reduce(static_cast<float>(count), a.tpr);
  const float inv_n = n_warp > 0.0f ? 1.0f / n_warp : 0.0f;
  float n_other = 0.0f, inv_other = 0.0f;  // of the warp that exchange() hands over
  if (a.tpr > 32) {
    const float2 other = exchange(make_float2(n_warp, inv_n), a.tpr, red[1]);
    n_other = other.x, inv_other = other.y;
  }
  uint32_t stage = own, next = own + (S - 1) * stage_bytes;
  T* y = static_cast<T*>(a.y) + t * a.d;
  T* z_row = static_cast<T*>(a.z) + t * a.d;
  for (int64_t round = 0; round < rounds; ++round) {
    fetch(next);
    copy_wait<S - 1>();
    const bool live = t < a.T;
    float2 v[kChunks * P], s = both(0.0f);
    if (live) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (!at.any(c)) continue;
        uint4 u = load_slot(stage + c * kPitch);
        if (res) {
          // the sum is rounded to the rows' type here: it is what the caller
          // keeps and what the backward normalises again
          u = add_chunks<T>(u, load_slot(stage + (kChunks + c) * kPitch));
          at.store(z_row, c, u);
        }
        unpack_pairs<T>(u, v + c * P);
        at.mask(c, v + c * P, 0.0f);
#pragma unroll
        for (int i = 0; i < P; ++i) s = add2(s, v[c * P + i]);
      }
    }
    const float sum = warp_reduce(s.x + s.y, a.tpr);
    const float mid = sum * inv_n;  // the warp's mean
    s = both(0.0f);
    if (live) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (!at.any(c)) continue;
        at.mask(c, v + c * P, mid);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          float2& e = v[c * P + i];
          e = add2(e, both(-mid));
          s = fma2(e, e, s);
        }
      }
    }
    float q = warp_reduce(s.x + s.y, a.tpr), mu = mid;
    if (a.tpr > 32) {
      const float2 other = exchange(make_float2(sum, q), a.tpr, red[round & 1]);
      mu = over_warps(other.x, a.tpr >> 5) * inv_d;
      const float e = other.x * inv_other - mu;
      q = over_warps(fmaf(n_other * e, e, other.y), a.tpr >> 5);
    }
    const float r = rsqrtf(fmaf(q, inv_d, a.eps));
    if (live) {
      if (lane == 0) {
        a.stats[t] = mu;
        a.stats[a.T + t] = r;
      }
      const float2 r2 = both(r), shift = both((mid - mu) * r);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (!at.any(c)) continue;
        // (z - mu) r = (z - mid) r + (mid - mu) r
#pragma unroll
        for (int i = 0; i < P; ++i)
          v[c * P + i] = fma2(fma2(v[c * P + i], r2, shift), w[c * P + i], b[c * P + i]);
        at.store(y, c, pack_pairs<T>(v + c * P));
      }
    }
    t += step;
    y += step * a.d;
    if (res) z_row += step * a.d;
    next = stage;
    stage = stage + stage_bytes == own + S * stage_bytes ? own : stage + stage_bytes;
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
  const float r = rsqrtf(group_reduce(s, a.tpr, red[1]) * inv_d + a.eps);
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
  const float r = rsqrtf(group_reduce(s, blockDim.x, red[1]) / static_cast<float>(a.d) + a.eps);
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

// The block's column sums from its threads': where the lanes of a warp own
// the same columns (`same`: tpr below 32, rows that start alike) they add by
// a tree, then the warps or groups in order through `shared` (slots x d
// floats).  column(i): value i's column.  In a cluster the block's sums stay
// in shared memory behind the slots, 2 x d floats.
__device__ __forceinline__ float* cluster_sums(const BackwardArgs& a, bool same, float* shared) {
  const int slots = blockDim.x / (same && a.tpr < 32 ? 32 : a.tpr);
  return shared + (slots > 1 ? slots * a.d : 0);
}

// dw and db from the sums of a cluster's blocks: each block takes every
// cluster-th run of threads' columns and adds the blocks' sums in order.
__device__ __forceinline__ void finish_cluster(const BackwardArgs& a, bool same, float* shared) {
  const float* sums = cluster_sums(a, same, shared);
  cluster_sync();
  for (int which = 0; which < 2; ++which) {
    float* out = which ? a.db : a.dw;
    if (!out) continue;
    for (int j = cluster_rank() * blockDim.x + threadIdx.x; j < a.d; j += a.cluster * blockDim.x) {
      float s = 0.0f;
      for (int k = 0; k < a.cluster; ++k) s += remote_f32(sums + which * a.d + j, k);
      out[j] = s;
    }
  }
  cluster_sync();  // no block leaves while another reads its sums
}

template <int kValues, typename Value, typename Column>
__device__ __forceinline__ void write_partial(const BackwardArgs& a, int which, bool same, float* shared, Value value,
                                              Column column) {
  const int tpr = a.tpr, d = a.d;
  const int width = same && tpr < 32 ? 32 : tpr;  // threads whose sums share a slot
  const int slots = blockDim.x / width, slot = threadIdx.x / width;
  const bool owner = threadIdx.x % width < tpr;
  float* out = a.cluster ? cluster_sums(a, same, shared) + which * d
                         : a.partial + (static_cast<int64_t>(blockIdx.x) * 2 + which) * d;
  __syncthreads();  // the ring, or the other sum, is done with `shared`
#pragma unroll
  for (int i = 0; i < kValues; ++i) {
    float s = value(i);
    for (int k = width >> 1; k >= tpr; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    const int j = column(i);
    if (owner && j >= 0 && j < d) (slots == 1 ? out : shared + slot * d)[j] = s;
  }
  if (slots == 1) return;
  __syncthreads();
  for (int j = threadIdx.x; j < d; j += blockDim.x) {
    float s = shared[j];
    for (int k = 1; k < slots; ++k) s += shared[k * d + j];
    out[j] = s;
  }
}

template <typename T, int kChunks, bool kAligned>
__global__ void __launch_bounds__(kRingThreads, 1) backward_ring_kernel(const BackwardArgs a) {
  constexpr int P = kPairs<T>, S = kBackwardStages<kChunks>;
  constexpr bool kKeep = kChunks * P <= 8;  // at most 16 values a thread
  extern __shared__ uint4 ring[];  // [stage][operand][chunk][thread]
  __shared__ float2 red[2][kMaxWarps];
  let_next_start();
  const int groups = kRingThreads / a.tpr, lane = threadIdx.x % a.tpr;
  const bool add = a.dz.ptr != nullptr;
  const uint32_t own = smem_addr(ring) + threadIdx.x * 16, stage_bytes = (add ? 3 : 2) * kChunks * kPitch;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups;
  const int64_t rounds = (a.T - first + step - 1) / step;
  int64_t t = first + threadIdx.x / a.tpr;
  const Place<T, kChunks, kAligned> at(lane, a.tpr, a.d, kAligned ? 0 : row_offset<T>(a.dy, t));
  const T* dy = static_cast<const T*>(a.dy.ptr) + t * a.dy.stride;
  const T* z = static_cast<const T*>(a.z.ptr) + t * a.z.stride;
  const T* dz = static_cast<const T*>(a.dz.ptr) + (add ? t * a.dz.stride : 0);
  int64_t ahead = t;  // the row that the pointers stand at
  auto fetch = [&](uint32_t stage) {
    if (ahead < a.T) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (!at.any(c)) continue;
        at.fetch(stage + c * kPitch, dy, c);
        at.fetch(stage + (kChunks + c) * kPitch, z, c);
        if (add) at.fetch(stage + (2 * kChunks + c) * kPitch, dz, c);
      }
    }
    copy_commit();
    ahead += step;
    dy += step * a.dy.stride;
    z += step * a.z.stride;
    if (add) dz += step * a.dz.stride;
  };
  for (int s = 0; s < S - 1; ++s) fetch(own + s * stage_bytes);
  float2 w[kChunks * P], sw[kChunks * P], sb[kChunks * P];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) at.params(c, a.w, a.w_f32, 1.0f, w + c * P);
#pragma unroll
  for (int i = 0; i < kChunks * P; ++i) sw[i] = sb[i] = both(0.0f);
  const float inv_d = 1.0f / static_cast<float>(a.d);
  uint32_t stage = own, next = own + (S - 1) * stage_bytes;
  T* dx = static_cast<T*>(a.dx) + t * a.d;
  float mu = 0.0f, r = 0.0f;
  if (t < a.T) mu = __ldg(a.stats + t), r = __ldg(a.stats + a.T + t);
  for (int64_t round = 0; round < rounds; ++round) {
    fetch(next);
    float next_mu = 0.0f, next_r = 0.0f;
    if (t + step < a.T) next_mu = __ldg(a.stats + t + step), next_r = __ldg(a.stats + a.T + t + step);
    copy_wait<S - 1>();
    const bool live = t < a.T;
    const float2 m2 = both(-mu), r2 = both(r);
    float2 s1 = both(0.0f), s2 = both(0.0f);
    // the row's n and g w, kept over the exchange where the registers hold
    // them beside the column sums, else made again from the slots
    float2 n_row[kKeep ? kChunks * P : 1], gw_row[kKeep ? kChunks * P : 1];
    if (live) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (!at.any(c)) continue;
        float2 g[P], n[P];
        unpack_pairs<T>(load_slot(stage + c * kPitch), g);
        unpack_pairs<T>(load_slot(stage + (kChunks + c) * kPitch), n);
        at.mask(c, g, 0.0f);
        at.mask(c, n, mu);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          n[i] = mul2(add2(n[i], m2), r2);
          sw[c * P + i] = fma2(g[i], n[i], sw[c * P + i]);
          sb[c * P + i] = add2(g[i], sb[c * P + i]);
          g[i] = mul2(g[i], w[c * P + i]);
          s1 = add2(s1, g[i]);
          s2 = fma2(g[i], n[i], s2);
          if (kKeep) {
            n_row[kKeep ? c * P + i : 0] = n[i];
            gw_row[kKeep ? c * P + i : 0] = g[i];
          }
        }
      }
    }
    const float2 sum = group_reduce(make_float2(s1.x + s1.y, s2.x + s2.y), a.tpr, red[round & 1]);
    if (live) {
      const float2 m1 = both(-sum.x * inv_d), c2 = both(-sum.y * inv_d);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (!at.any(c)) continue;
        float2 g[P], n[P];
        if (kKeep) {
#pragma unroll
          for (int i = 0; i < P; ++i)
            g[i] = fma2(n_row[kKeep ? c * P + i : 0], c2, add2(gw_row[kKeep ? c * P + i : 0], m1));
        } else {
          unpack_pairs<T>(load_slot(stage + c * kPitch), g);
          unpack_pairs<T>(load_slot(stage + (kChunks + c) * kPitch), n);
#pragma unroll
          for (int i = 0; i < P; ++i)
            g[i] = fma2(mul2(add2(n[i], m2), r2), c2, fma2(g[i], w[c * P + i], m1));
        }
        if (add) {
          unpack_pairs<T>(load_slot(stage + (2 * kChunks + c) * kPitch), n);
#pragma unroll
          for (int i = 0; i < P; ++i) g[i] = fma2(g[i], r2, n[i]);
        } else {
#pragma unroll
          for (int i = 0; i < P; ++i) g[i] = mul2(g[i], r2);
        }
        at.store(dx, c, pack_pairs<T>(g));
      }
    }
    t += step;
    dx += step * a.d;
    mu = next_mu;
    r = next_r;
    next = stage;
    stage = stage + stage_bytes == own + S * stage_bytes ? own : stage + stage_bytes;
  }
  auto column = [&](int i) { return at.j0[i / (2 * P)] + i % (2 * P); };
  auto part = [](const float2* v, int i) { return i & 1 ? v[i >> 1].y : v[i >> 1].x; };
  float* shared = reinterpret_cast<float*>(ring);
  if (a.want_w)
    write_partial<kChunks * 2 * P>(a, 0, kAligned, shared, [&](int i) { return part(sw, i); }, column);
  if (a.want_b)
    write_partial<kChunks * 2 * P>(a, 1, kAligned, shared, [&](int i) { return part(sb, i); }, column);
  if (a.cluster) finish_cluster(a, kAligned, shared);
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
  auto column = [&](int i) { return lane + i * a.tpr; };
  float* shared = reinterpret_cast<float*>(ring);
  if (a.want_w) write_partial<kValues>(a, 0, true, shared, [&](int i) { return sw[i]; }, column);
  if (a.want_b) write_partial<kValues>(a, 1, true, shared, [&](int i) { return sb[i]; }, column);
  if (a.cluster) finish_cluster(a, true, shared);
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
// Threads (a power of two) for a row of `units` chunks or values: up to a
// warp, one each; then as few as hold the row with `most` each.
int threads_per_row(int units, int most) {
  int tpr = 1;
  while (tpr < 32 && tpr < units) tpr *= 2;
  while (tpr * most < units) tpr *= 2;
  return tpr;
}

int grid_of(int64_t T, int groups, int most) {
  const int64_t want = (T + groups - 1) / groups;
  return static_cast<int>(want < most ? want : most);
}

// Blocks of a ring kernel: one an SM.  With rows that do not start on a
// chunk, all blocks together take a multiple of `values` rows a round
// (`values` is a power of two, and so is the number of groups).
int ring_grid(int64_t T, int tpr, int values, bool aligned, int num_sms) {
  const int groups = kRingThreads / tpr;
  const int multiple = aligned || groups >= values ? 1 : values / groups;
  const int grid = grid_of(T, groups, num_sms);
  const int up = (grid + multiple - 1) / multiple * multiple;
  return up <= num_sms ? up : num_sms / multiple * multiple;
}

template <typename T, int kChunks, bool kAligned>
cudaError_t forward_ring(const ForwardArgs& a, int num_sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr size_t operand = static_cast<size_t>(kForwardStages<kChunks>) * kChunks * kPitch;
  const cudaError_t err =
      allow(reinterpret_cast<const void*>(forward_ring_kernel<T, kChunks, kAligned>), done, 2 * operand, false);
  if (err != cudaSuccess) return err;
  forward_ring_kernel<T, kChunks, kAligned>
      <<<ring_grid(a.T, a.tpr, kChunk<T>, kAligned, num_sms), kRingThreads, (a.res.ptr ? 2 : 1) * operand, stream>>>(a);
  return cudaGetLastError();
}

// How rows lie: on chunks, or all alike within 16 bytes, or neither.  Each
// operand's base and row stride in bytes.
struct Lie {
  bool on_chunks = true, alike = true;
  uintptr_t base0;
  int64_t stride0;
  Lie(const void* p, int64_t stride_bytes) : base0(reinterpret_cast<uintptr_t>(p)), stride0(stride_bytes) {
    add(p, stride_bytes);
  }
  void add(const void* p, int64_t stride_bytes) {
    const uintptr_t base = reinterpret_cast<uintptr_t>(p);
    if (base % 16 != 0 || stride_bytes % 16 != 0) on_chunks = false;
    if ((base - base0) % 16 != 0 || (stride_bytes - stride0) % 16 != 0) alike = false;
  }
};

bool param_on_chunks(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Threads for a ring's row, or 0 where 3 chunks a thread do not hold it.  A
// row that does not start on a chunk may touch one more than it fills, and
// has at least 8 threads (its groups' column sums are added one by one).
int ring_threads(int d, int values, bool aligned, int* per_thread) {
  const int chunks = (d + values - 1) / values + (aligned ? 0 : 1);
  int tpr = threads_per_row(chunks, 3);
  if (!aligned && tpr < 8) tpr = 8;
  *per_thread = (chunks + tpr - 1) / tpr;
  return tpr <= kRingThreads ? tpr : 0;
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
  Lie lie(a.x.ptr, a.T > 1 ? a.x.stride * e : a.d * e);
  lie.add(a.y, static_cast<int64_t>(a.d) * e);
  if (a.res.ptr) {
    lie.add(a.res.ptr, a.T > 1 ? a.res.stride * e : a.d * e);
    lie.add(a.z, static_cast<int64_t>(a.d) * e);
  }
  const bool aligned = lie.on_chunks && a.d % N == 0 && param_on_chunks(a.w) && param_on_chunks(a.b);
  int per_thread = 0;
  if (aligned || lie.alike) a.tpr = ring_threads(a.d, N, aligned, &per_thread);
  if (a.tpr > 0) {
    if (aligned) {
      if (per_thread == 1) return forward_ring<T, 1, true>(a, num_sms, stream);
      if (per_thread == 2) return forward_ring<T, 2, true>(a, num_sms, stream);
      return forward_ring<T, 3, true>(a, num_sms, stream);
    }
    if (per_thread == 1) return forward_ring<T, 1, false>(a, num_sms, stream);
    if (per_thread == 2) return forward_ring<T, 2, false>(a, num_sms, stream);
    return forward_ring<T, 3, false>(a, num_sms, stream);
  }
  // at most 8 values a thread: more spill at 1,024 threads
  a.tpr = threads_per_row(a.d, 8);
  if (a.tpr <= 1024)
    return a.d <= a.tpr * 4 ? forward_values<T, 4>(a, stream) : forward_values<T, 8>(a, stream);
  forward_long_kernel<T><<<static_cast<unsigned>(a.T), 1024, 0, stream>>>(a);
  return cudaGetLastError();
}

// Blocks of the one cluster that takes T rows, or 0 where they are more than
// 2 rounds of the largest (further rounds cost more than the second launch
// that the cluster saves: 160 x 2816 in 3 rounds 11.3 us on the GPU, as two
// launches 7.9 us).
int cluster_blocks(int64_t T, int groups, int multiple) {
  if (T > static_cast<int64_t>(groups) * kClusterMost * 2) return 0;
  const int want = grid_of(T, groups, kClusterMost);
  int blocks = 1;
  while (blocks < want || blocks % multiple != 0) blocks *= 2;
  return blocks;
}

template <typename T, int kChunks, bool kAligned>
cudaError_t backward_ring(BackwardArgs& a, int num_sms, int* blocks, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr size_t operand = static_cast<size_t>(kBackwardStages<kChunks>) * kChunks * kPitch;
  const cudaError_t err =
      allow(reinterpret_cast<const void*>(backward_ring_kernel<T, kChunks, kAligned>), done, 3 * operand, true);
  if (err != cudaSuccess) return err;
  const size_t smem = (a.dz.ptr ? 3 : 2) * operand;
  const int groups = kRingThreads / a.tpr;
  const int multiple = kAligned || groups >= kChunk<T> ? 1 : kChunk<T> / groups;
  a.cluster = cluster_blocks(a.T, groups, multiple);
  if (a.cluster)
    return launch_cluster(backward_ring_kernel<T, kChunks, kAligned>, a.cluster, kRingThreads, smem, stream, a);
  *blocks = ring_grid(a.T, a.tpr, kChunk<T>, kAligned, num_sms);
  backward_ring_kernel<T, kChunks, kAligned><<<*blocks, kRingThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, int kValues>
cudaError_t backward_values(BackwardArgs& a, int num_sms, int* blocks, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const int block = a.tpr < 256 ? 256 : a.tpr, groups = block / a.tpr;
  const int slots = a.tpr < 32 ? block / 32 : groups;
  size_t smem = slots > 1 ? static_cast<size_t>(slots) * a.d * 4 : 0;  // at most 8 x 256 floats
  a.cluster = cluster_blocks(a.T, groups, 1);
  if (a.cluster) {
    smem += static_cast<size_t>(2) * a.d * 4;
    const cudaError_t err = allow(reinterpret_cast<const void*>(backward_values_kernel<T, kValues>), done,
                                  static_cast<size_t>(8 * 256 + 2 * kRingThreads * kValues) * 4, true);
    if (err != cudaSuccess) return err;
    return launch_cluster(backward_values_kernel<T, kValues>, a.cluster, block, smem, stream, a);
  }
  const int most = num_sms * (kRingThreads / block);
  *blocks = grid_of(a.T, groups, most < kNormMaxBlocks ? most : kNormMaxBlocks);
  backward_values_kernel<T, kValues><<<*blocks, block, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward_typed(BackwardArgs& a, int num_sms, int* blocks, cudaStream_t stream) {
  constexpr int N = kChunk<T>, e = sizeof(T);
  Lie lie(a.dy.ptr, a.T > 1 ? a.dy.stride * e : a.d * e);
  lie.add(a.z.ptr, a.T > 1 ? a.z.stride * e : a.d * e);
  if (a.dz.ptr) lie.add(a.dz.ptr, a.T > 1 ? a.dz.stride * e : a.d * e);
  lie.add(a.dx, static_cast<int64_t>(a.d) * e);
  const bool aligned = lie.on_chunks && a.d % N == 0 && param_on_chunks(a.w);
  int per_thread = 0;
  if (aligned || lie.alike) a.tpr = ring_threads(a.d, N, aligned, &per_thread);
  if (a.tpr > 0) {
    if (aligned) {
      if (per_thread == 1) return backward_ring<T, 1, true>(a, num_sms, blocks, stream);
      if (per_thread == 2) return backward_ring<T, 2, true>(a, num_sms, blocks, stream);
      return backward_ring<T, 3, true>(a, num_sms, blocks, stream);
    }
    if (per_thread == 1) return backward_ring<T, 1, false>(a, num_sms, blocks, stream);
    if (per_thread == 2) return backward_ring<T, 2, false>(a, num_sms, blocks, stream);
    return backward_ring<T, 3, false>(a, num_sms, blocks, stream);
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
                 f.weight_dtype == MOE_F32, f.T, f.d, f.dx, f.partial, f.dweight, f.dbias, f.dweight != nullptr,
                 f.dbias != nullptr, 0, 0};
  int blocks = 0;
  cudaError_t err;
  switch (f.dtype) {
    case MOE_F32: err = backward_typed<float>(a, num_sms, &blocks, stream); break;
    case MOE_BF16: err = backward_typed<__nv_bfloat16>(a, num_sms, &blocks, stream); break;
    default: err = backward_typed<__half>(a, num_sms, &blocks, stream); break;
  }
  if (err != cudaSuccess || a.cluster || !(a.want_w || a.want_b)) return err;
  return launch_dependent(finish_kernel, dim3((f.d + 31) / 32, 2), 1024, 0, stream, f.partial, blocks, f.d, f.dweight,
                          f.dbias);
}

}  // namespace moe
