// Layer norm over the rows of [T, d], forward (layer_norm_forward.cuh) and
// backward (layer_norm_backward.cuh): what both share.
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
//     16 bytes (contiguous tensors of any d do) and 4 chunks a thread of 512
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
//   - rows longer than that: a block a row that keeps the row in shared
//     memory where it fits (else the later sweeps read it again).
// The variance is taken from the deviations from the mean, never as a
// difference of two sums, so a large common offset costs no digits.  Sums
// are fp32 per thread and then trees over lanes and warps, always in the same
// order.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "internal.h"
#include "launch.cuh"

namespace moe {

struct NormRows {
  const void* ptr;
  int64_t stride;  // elements between rows
};

struct NormForwardArgs {
  NormRows x, res;
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
  int tile_rounds;  // rounds of a block's piece of work
  int64_t piece;    // its rows
  bool steal;       // more pieces than SMs
};

struct NormBackwardArgs {
  NormRows dy, z, dz;
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

// One translation unit for each element type (layer_norm_f32.cu, _bf16.cu,
// _f16.cu).  The backward sets *blocks to the number of partial sums it left,
// or a.cluster where it left none.
template <typename T>
cudaError_t norm_forward_typed(NormForwardArgs& a, int num_sms, cudaStream_t stream);
template <typename T>
cudaError_t norm_backward_typed(NormBackwardArgs& a, int num_sms, int* blocks, cudaStream_t stream);

namespace {

using Row = NormRows;
using ForwardArgs = NormForwardArgs;
using BackwardArgs = NormBackwardArgs;

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

// Hands each warp's values to the whole group: the calling lane gets those of
// warp lane mod warps.  `red` is one of two buffers used in turn: a thread
// reaches the next exchange's barrier only after it has read this one's
// buffer, so one barrier each is enough.
template <int kRows>
__device__ __forceinline__ void exchange(float2 (&v)[kRows], int tpr, int group, float2* red) {
  const int lane = threadIdx.x & 31, warps = tpr >> 5;
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    if (lane == i) red[i * kMaxWarps + (threadIdx.x >> 5)] = v[i];
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
#pragma unroll
  for (int i = 0; i < kRows; ++i) v[i] = red[i * kMaxWarps + group * warps + (lane & (warps - 1))];
}
__device__ __forceinline__ float2 exchange(float2 v, int tpr, int group, float2* red) {
  float2 a[1] = {v};
  exchange(a, tpr, group, red);
  return a[0];
}

// Sums over the row's group, in every thread of it.
__device__ __forceinline__ float2 group_reduce(float2 v, int tpr, float2* red) {
  v = warp_reduce(v, tpr);
  return tpr <= 32 ? v : over_warps(exchange(v, tpr, threadIdx.x / tpr, red), tpr >> 5);
}

__device__ __forceinline__ float group_reduce(float v, int tpr, float2* red) {
  v = warp_reduce(v, tpr);
  return tpr <= 32 ? v : over_warps(exchange(make_float2(v, 0.0f), tpr, threadIdx.x / tpr, red).x, tpr >> 5);
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
// 512 threads an SM, at most 128 registers each.
constexpr int kRingThreads = 512;

// How a row fits its threads' chunks: it starts anywhere; on a chunk; or on a
// chunk and fills every chunk of every thread (nothing to check).
enum Fit { kAnywhere, kOnChunks, kFull };

// Where a thread's chunks lie, for all of its rows.
template <typename T, int kChunks, Fit kFit>
struct Place {
  static constexpr int N = kChunk<T>;
  static constexpr bool kAligned = kFit != kAnywhere;
  int j0[kChunks];  // first column of each chunk: from -off up, at least d for a chunk beyond the row
  int d;
  __device__ __forceinline__ Place(int lane, int tpr, int d_, int off) : d(d_) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) j0[c] = (lane + c * tpr) * N - (kAligned ? 0 : off);
  }
  __device__ __forceinline__ bool any(int c) const { return kFit == kFull || j0[c] < d; }
  __device__ __forceinline__ bool whole(int c) const { return kAligned || (j0[c] >= 0 && j0[c] + N <= d); }
  // Copies the chunk.  A partial first chunk is copied whole: its 16 aligned
  // bytes hold at least one value of the row, so they lie inside the
  // row's allocation.  A last chunk ends with the row.
  __device__ __forceinline__ void fetch(uint32_t slot, const T* row, int c) const {
    if (kAligned || j0[c] + N <= d) copy_async(slot, row + j0[c]);
    else copy_async_part(slot, row + j0[c], (d - j0[c]) * static_cast<int>(sizeof(T)));
  }
  // The chunk in its slot; zeros where the row does not reach it.
  __device__ __forceinline__ uint4 load(uint32_t slot, int c) const {
    return any(c) ? load_slot(slot) : make_uint4(0, 0, 0, 0);
  }
  // Values outside the row become `fill`.
  __device__ __forceinline__ void mask(int c, float2* v, float fill) const {
    if (kFit == kFull || (kAligned ? any(c) : whole(c))) return;
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

// ---- long rows: units of a chunk (kVec) or of one value
template <typename T, bool kVec>
struct Unit {
  static constexpr int N = kVec ? kChunk<T> : 1;
  using Store = typename std::conditional<kVec, uint4, T>::type;
  __device__ static __forceinline__ void values(const Store& u, float* v) {
    if constexpr (kVec) unpack_chunk<T>(u, v);
    else v[0] = to_f32(u);
  }
  __device__ static __forceinline__ Store store(const float* v) {
    if constexpr (kVec) return pack_chunk<T>(v);
    else return from_f32<T>(v[0]);
  }
  __device__ static __forceinline__ void params(const void* p, bool f32, float missing, int u, float* v) {
    if (!p) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = missing;
    } else if constexpr (!kVec) {
      v[0] = param_at<T>(p, f32, u);
    } else if (f32) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        *reinterpret_cast<float4*>(v + i) = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + u * N + i));
    } else {
      unpack_chunk<T>(__ldg(static_cast<const uint4*>(p) + u), v);
    }
  }
};
constexpr size_t kLongCache = 200 * 1024;  // shared memory for a long row

template <typename T>
__device__ __forceinline__ int row_offset(const Row& rows, int64_t t) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(static_cast<const T*>(rows.ptr) + t * rows.stride) & 15) /
                          sizeof(T));
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

// Blocks of a ring kernel with `groups` groups each, `resident` at a time:
// never more than there are rows, which is what the backward's workspace holds
// partial sums for.  A block for each of its groups' rows where they are few
// enough: no group then has a second row.  Else, with rows that do not start
// on a chunk, all blocks together take a multiple of `values` rows a round
// (`values` is a power of two, and so is `groups`).
int ring_grid(int64_t T, int groups, int values, bool aligned, int resident) {
  const int grid = grid_of(T, groups, resident);
  const int multiple = aligned || groups >= values ? 1 : values / groups;
  return grid < resident ? grid : resident / multiple * multiple;
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

// Threads for a ring's row, or 0 where 4 chunks a thread do not hold it (4 for
// the longest rows only: their registers spill a little).  A
// row that does not start on a chunk may touch one more than it fills, and
// has at least 8 threads (its groups' column sums are added one by one).
int ring_threads(int d, int values, bool aligned, int* per_thread) {
  const int chunks = (d + values - 1) / values + (aligned ? 0 : 1);
  int tpr = threads_per_row(chunks, 3);
  if (!aligned && tpr < 8) tpr = 8;
  if (tpr > kRingThreads && chunks <= 4 * kRingThreads) tpr = kRingThreads;
  *per_thread = (chunks + tpr - 1) / tpr;
  return tpr <= kRingThreads ? tpr : 0;
}

}  // namespace
}  // namespace moe
