// Layer norm over the rows of [T, d], forward and backward.
//
//   z  = round(x + residual)  (or x)          mu = mean z
//   r  = 1 / sqrt(mean (z - mu)^2 + eps)      n  = (z - mu) r
//   y  = round(n w + b)
// and for an output gradient dy, g = dy w:
//   dx = r (g - mean g - n mean(g n)) + dz    dw = sum_t dy n    db = sum_t dy
//
// A row belongs to a group of `tpr` threads (a power of two); thread i of the
// group owns the 16-byte chunks i, i + tpr, ... of the row and keeps them in
// registers, so a row is read once.  The variance is taken from the
// deviations from the mean, never as a difference of two sums, so a large
// common offset costs no digits.  Sums are fp32 per thread and then trees
// over lanes and warps, always in the same order.
#include "common.cuh"
#include "elem.cuh"
#include "internal.h"

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
  bool same_phase;  // unaligned rows: every operand has the row's position within 16 bytes
};

// Sum over the row's group, in every thread of it; `red` holds two sets of
// 32 floats used in turn, so one barrier a sum is enough.
__device__ __forceinline__ float row_sum(float v, int tpr, float* red) {
  if (tpr <= 32) return group_sum(v, tpr);
  v = group_sum(v, 32);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < (tpr >> 5) ? red[lane] : 0.0f;
  return group_sum(v, 32);
}

// Values [j0, j0 + N) of a row, zero outside [0, d).  kAligned: whole chunks
// at 16-byte addresses; otherwise the first and the last chunk of a row may
// be partial and are read value by value, as is every chunk of an operand
// that lies differently within 16 bytes (`vec` false).
template <typename T, bool kAligned>
__device__ __forceinline__ uint4 load_chunk(const T* row, int j0, int d, bool vec) {
  constexpr int N = kChunk<T>;
  if (kAligned || (vec && j0 >= 0 && j0 + N <= d)) return __ldg(reinterpret_cast<const uint4*>(row + j0));
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (j0 + i >= 0 && j0 + i < d) ? to_f32(row[j0 + i]) : 0.0f;
  return pack_chunk<T>(v);
}

template <typename T, bool kAligned>
__device__ __forceinline__ void store_chunk(T* row, int j0, int d, bool vec, const float* v) {
  constexpr int N = kChunk<T>;
  if (kAligned || (vec && j0 >= 0 && j0 + N <= d)) {
    *reinterpret_cast<uint4*>(row + j0) = pack_chunk<T>(v);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (j0 + i >= 0 && j0 + i < d) row[j0 + i] = from_f32<T>(v[i]);
}

// N values of the weight or the bias at columns j0.. (fp32 or of type T).
template <typename T, bool kAligned>
__device__ __forceinline__ void load_param(const void* p, bool f32, int j0, int d, float* v) {
  constexpr int N = kChunk<T>;
  if (kAligned) {
    if (f32) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        *reinterpret_cast<float4*>(v + i) = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + j0 + i));
    } else {
      unpack_chunk<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p) + j0)), v);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int j = j0 + i;
    v[i] = 0.0f;
    if (j >= 0 && j < d) v[i] = f32 ? __ldg(static_cast<const float*>(p) + j) : to_f32(static_cast<const T*>(p)[j]);
  }
}

// Elements by which a row starts after a 16-byte boundary.
template <typename T>
__device__ __forceinline__ int row_phase(const T* p) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
}

template <typename T, int kChunks, bool kAligned>
__global__ void __launch_bounds__(1024) forward_kernel(const ForwardArgs a) {
  constexpr int N = kChunk<T>;
  __shared__ float red[2][32];
  const int groups = blockDim.x / a.tpr, lane = threadIdx.x % a.tpr;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / a.tpr;
  const bool live = t < a.T;  // groups beyond the last row follow along without memory accesses
  const int64_t row = live ? t : 0;
  const T* x = static_cast<const T*>(a.x.ptr) + row * a.x.stride;
  const T* res = static_cast<const T*>(a.res.ptr) + (a.res.ptr ? row * a.res.stride : 0);
  const int off = kAligned ? 0 : row_phase(x);
  const int d = live ? a.d : 0;
  uint4 raw[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int j0 = (lane + c * a.tpr) * N - off;
    raw[c] = make_uint4(0, 0, 0, 0);
    if (j0 < d) raw[c] = load_chunk<T, kAligned>(x, j0, d, true);
  }
  if (a.res.ptr) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int j0 = (lane + c * a.tpr) * N - off;
      if (j0 < d) {
        float u[N], v[N];
        unpack_chunk<T>(raw[c], u);
        unpack_chunk<T>(load_chunk<T, kAligned>(res, j0, d, a.same_phase), v);
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] += v[i];
        // the sum is rounded to the rows' type here: it is what the caller
        // keeps and what the backward normalises again
        raw[c] = pack_chunk<T>(u);
        store_chunk<T, kAligned>(static_cast<T*>(a.z) + row * a.d, j0, d, a.same_phase, u);
      }
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    float v[N];
    unpack_chunk<T>(raw[c], v);
#pragma unroll
    for (int i = 0; i < N; ++i) s += v[i];
  }
  const float mu = row_sum(s, a.tpr, red[0]) / static_cast<float>(a.d);
  s = 0.0f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int j0 = (lane + c * a.tpr) * N - off;
    float v[N];
    unpack_chunk<T>(raw[c], v);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float e = v[i] - mu;
      if (kAligned ? j0 < d : (j0 + i >= 0 && j0 + i < d)) s += e * e;
    }
  }
  const float r = 1.0f / sqrtf(row_sum(s, a.tpr, red[1]) / static_cast<float>(a.d) + a.eps);
  if (live && lane == 0) {
    a.stats[t] = mu;
    a.stats[a.T + t] = r;
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int j0 = (lane + c * a.tpr) * N - off;
    if (j0 >= d) continue;
    float v[N], p[N];
    unpack_chunk<T>(raw[c], v);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (v[i] - mu) * r;
    if (a.w) {
      load_param<T, kAligned>(a.w, a.w_f32, j0, d, p);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= p[i];
    }
    if (a.b) {
      load_param<T, kAligned>(a.b, a.w_f32, j0, d, p);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += p[i];
    }
    store_chunk<T, kAligned>(static_cast<T*>(a.y) + row * a.d, j0, d, a.same_phase, v);
  }
}

// Rows too long for the registers of one block: three sweeps over the row,
// the second and the third out of L2 (or L1), one value a thread.
template <typename T>
__global__ void __launch_bounds__(1024) forward_long_kernel(const ForwardArgs a) {
  __shared__ float red[2][32];
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
  const float mu = row_sum(s, blockDim.x, red[0]) / static_cast<float>(a.d);
  s = 0.0f;
  for (int j = threadIdx.x; j < a.d; j += blockDim.x) {
    const float e = to_f32(in[j]) - mu;
    s += e * e;
  }
  const float r = 1.0f / sqrtf(row_sum(s, blockDim.x, red[1]) / static_cast<float>(a.d) + a.eps);
  if (threadIdx.x == 0) {
    a.stats[t] = mu;
    a.stats[a.T + t] = r;
  }
  for (int j = threadIdx.x; j < a.d; j += blockDim.x) {
    float v = (to_f32(in[j]) - mu) * r;
    if (a.w) v *= a.w_f32 ? static_cast<const float*>(a.w)[j] : to_f32(static_cast<const T*>(a.w)[j]);
    if (a.b) v += a.w_f32 ? static_cast<const float*>(a.b)[j] : to_f32(static_cast<const T*>(a.b)[j]);
    static_cast<T*>(a.y)[t * a.d + j] = from_f32<T>(v);
  }
}

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
  bool same_phase;
};

// A block walks over rows blockIdx.x * groups + g, + gridDim.x * groups, ...
// and keeps the column sums of its chunks in registers; at the end the
// groups of the block add theirs in shared memory in group order.
template <typename T, int kChunks, bool kAligned>
__global__ void __launch_bounds__(512) backward_kernel(const BackwardArgs a) {
  constexpr int N = kChunk<T>;
  __shared__ float red[4][32];
  const int groups = blockDim.x / a.tpr, lane = threadIdx.x % a.tpr, group = threadIdx.x / a.tpr;
  float sw[kChunks * N], sb[kChunks * N];
#pragma unroll
  for (int i = 0; i < kChunks * N; ++i) sw[i] = sb[i] = 0.0f;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * groups; t0 < a.T;
       t0 += static_cast<int64_t>(gridDim.x) * groups) {
    const int64_t t = t0 + group;
    const bool live = t < a.T;
    const int64_t row = live ? t : 0;
    const int d = live ? a.d : 0;
    const T* dy = static_cast<const T*>(a.dy.ptr) + row * a.dy.stride;
    const T* z = static_cast<const T*>(a.z.ptr) + row * a.z.stride;
    const float mu = __ldg(a.stats + row), r = __ldg(a.stats + a.T + row);
    uint4 raw_dy[kChunks], raw_z[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int j0 = (lane + c * a.tpr) * N;
      raw_dy[c] = raw_z[c] = make_uint4(0, 0, 0, 0);
      if (j0 < d) {
        raw_dy[c] = load_chunk<T, kAligned>(dy, j0, d, false);
        raw_z[c] = load_chunk<T, kAligned>(z, j0, d, false);
      }
    }
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int j0 = (lane + c * a.tpr) * N;
      if (j0 >= d) continue;
      float g[N], n[N], p[N];
      unpack_chunk<T>(raw_dy[c], g);
      unpack_chunk<T>(raw_z[c], n);
      if (a.w) load_param<T, kAligned>(a.w, a.w_f32, j0, d, p);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        n[i] = (n[i] - mu) * r;
        sw[c * N + i] += g[i] * n[i];  // columns past d: their dy is zero
        sb[c * N + i] += g[i];
        const float gw = a.w ? g[i] * p[i] : g[i];
        s1 += gw;
        s2 += gw * n[i];
      }
    }
    if (a.tpr <= 32) {
      s1 = group_sum(s1, a.tpr);
      s2 = group_sum(s2, a.tpr);
    } else {
      s1 = row_sum(s1, a.tpr, red[0]);
      s2 = row_sum(s2, a.tpr, red[1]);
      __syncthreads();
    }
    s1 *= inv_d;
    s2 *= inv_d;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int j0 = (lane + c * a.tpr) * N;
      if (j0 >= d) continue;
      float g[N], n[N], p[N];
      unpack_chunk<T>(raw_dy[c], g);
      unpack_chunk<T>(raw_z[c], n);
      if (a.w) {
        load_param<T, kAligned>(a.w, a.w_f32, j0, d, p);
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] *= p[i];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        n[i] = (n[i] - mu) * r;
        g[i] = (g[i] - s1 - n[i] * s2) * r;
      }
      if (a.dz.ptr) {
        unpack_chunk<T>(load_chunk<T, kAligned>(static_cast<const T*>(a.dz.ptr) + row * a.dz.stride, j0, d, false), p);
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] += p[i];
      }
      store_chunk<T, kAligned>(static_cast<T*>(a.dx) + row * a.d, j0, d, false, g);
    }
  }
  // the block's column sums
  extern __shared__ float sums[];
  for (int which = 0; which < 2; ++which) {
    if (!(which ? a.want_b : a.want_w)) continue;
    float* out = a.partial + (static_cast<int64_t>(blockIdx.x) * 2 + which) * a.d;
    for (int g = 0; g < groups; ++g) {
      if (g == group) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int j = (lane + c * a.tpr) * N + i;
            const float v = which ? sb[c * N + i] : sw[c * N + i];
            if (j >= a.d) continue;
            if (groups == 1) {
              out[j] = v;
            } else {
              const float before = g ? sums[j] : 0.0f;
              if (g == groups - 1) out[j] = before + v;
              else sums[j] = before + v;
            }
          }
      }
      if (groups > 1) __syncthreads();
    }
  }
}

// Rows too long for the registers: dx by a block a row in two sweeps, and
// the column sums by a block for each 256 columns and slice of rows.
template <typename T>
__global__ void __launch_bounds__(1024) backward_long_kernel(const BackwardArgs a) {
  __shared__ float red[2][32];
  const int64_t t = blockIdx.x;
  const T* dy = static_cast<const T*>(a.dy.ptr) + t * a.dy.stride;
  const T* z = static_cast<const T*>(a.z.ptr) + t * a.z.stride;
  const float mu = a.stats[t], r = a.stats[a.T + t];
  auto weight = [&](int j) {
    return !a.w ? 1.0f : a.w_f32 ? static_cast<const float*>(a.w)[j] : to_f32(static_cast<const T*>(a.w)[j]);
  };
  float s1 = 0.0f, s2 = 0.0f;
  for (int j = threadIdx.x; j < a.d; j += blockDim.x) {
    const float g = to_f32(dy[j]) * weight(j);
    s1 += g;
    s2 += g * ((to_f32(z[j]) - mu) * r);
  }
  s1 = row_sum(s1, blockDim.x, red[0]) / static_cast<float>(a.d);
  s2 = row_sum(s2, blockDim.x, red[1]) / static_cast<float>(a.d);
  for (int j = threadIdx.x; j < a.d; j += blockDim.x) {
    const float n = (to_f32(z[j]) - mu) * r;
    float v = (to_f32(dy[j]) * weight(j) - s1 - n * s2) * r;
    if (a.dz.ptr) v += to_f32(static_cast<const T*>(a.dz.ptr)[t * a.dz.stride + j]);
    static_cast<T*>(a.dx)[t * a.d + j] = from_f32<T>(v);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) column_sums_kernel(const BackwardArgs a, int slices) {
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

// dw and db: the blocks' sums added in block order, eight interleaved
// partial sums a column.
__global__ void __launch_bounds__(256) finish_kernel(const float* __restrict__ partial, int blocks, int d,
                                                     float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float part[8][32];
  const int j = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  float* out = blockIdx.y ? db : dw;
  if (out == nullptr) return;
  float s = 0.0f;
  if (j < d)
    for (int b = slice; b < blocks; b += 8) s += partial[(static_cast<int64_t>(b) * 2 + blockIdx.y) * d + j];
  part[slice][threadIdx.x & 31] = s;
  __syncthreads();
  if (slice == 0 && j < d) {
    for (int i = 1; i < 8; ++i) s += part[i][threadIdx.x];
    out[j] = s;
  }
}

bool chunk_aligned(const void* p, int64_t stride, int64_t T, int esize) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (T <= 1 || (stride * esize) % 16 == 0);
}

// Threads (a power of two) for a row of `chunks` chunks: up to a warp, one
// chunk each; then as few as hold the row with `most` chunks each.
int threads_per_row(int chunks, int most) {
  int tpr = 1;
  while (tpr < 32 && tpr < chunks) tpr *= 2;
  while (tpr * most < chunks) tpr *= 2;
  return tpr;
}

template <typename T, bool kAligned>
cudaError_t forward_launch(ForwardArgs& a, int per_thread, int block, cudaStream_t stream) {
  const int64_t grid = (a.T + block / a.tpr - 1) / (block / a.tpr);
  const unsigned g = static_cast<unsigned>(grid);
  switch (per_thread) {
    case 1: forward_kernel<T, 1, kAligned><<<g, block, 0, stream>>>(a); break;
    case 2: forward_kernel<T, 2, kAligned><<<g, block, 0, stream>>>(a); break;
    case 3: forward_kernel<T, 3, kAligned><<<g, block, 0, stream>>>(a); break;
    default: forward_kernel<T, 4, kAligned><<<g, block, 0, stream>>>(a); break;
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t forward_typed(ForwardArgs& a, cudaStream_t stream) {
  constexpr int N = kChunk<T>, e = sizeof(T);
  const int wsize = a.w_f32 ? 4 : e;
  const bool aligned = a.d % N == 0 && chunk_aligned(a.x.ptr, a.x.stride, a.T, e) &&
                       (!a.res.ptr || chunk_aligned(a.res.ptr, a.res.stride, a.T, e)) &&
                       chunk_aligned(a.y, a.d, a.T, e) && (!a.z || chunk_aligned(a.z, a.d, a.T, e)) &&
                       chunk_aligned(a.w, 0, 1, wsize) && chunk_aligned(a.b, 0, 1, wsize);
  // an unaligned row may touch one chunk more than it fills
  const int chunks = (a.d + N - 1) / N + (aligned ? 0 : 1);
  a.tpr = threads_per_row(chunks, 4);
  if (a.tpr > 1024) {
    forward_long_kernel<T><<<static_cast<unsigned>(a.T), 1024, 0, stream>>>(a);
    return cudaGetLastError();
  }
  const int per_thread = (chunks + a.tpr - 1) / a.tpr;
  const int block = a.tpr < 64 ? 128 : a.tpr;
  if (aligned) return forward_launch<T, true>(a, per_thread, block, stream);
  auto phase = [](const void* p) { return reinterpret_cast<uintptr_t>(p) & 15; };
  const bool rows_alike = a.T <= 1 || (a.x.stride - a.d) * e % 16 == 0;
  a.same_phase = rows_alike && phase(a.y) == phase(a.x.ptr) &&
                 (!a.res.ptr || (phase(a.res.ptr) == phase(a.x.ptr) && phase(a.z) == phase(a.x.ptr) &&
                                 (a.T <= 1 || (a.res.stride - a.x.stride) * e % 16 == 0)));
  return forward_launch<T, false>(a, per_thread, block, stream);
}

template <typename T, bool kAligned>
cudaError_t backward_launch(BackwardArgs& a, int per_thread, int block, int grid, size_t smem, cudaStream_t stream) {
  switch (per_thread) {
    case 1: backward_kernel<T, 1, kAligned><<<grid, block, smem, stream>>>(a); break;
    case 2: backward_kernel<T, 2, kAligned><<<grid, block, smem, stream>>>(a); break;
    default: backward_kernel<T, 3, kAligned><<<grid, block, smem, stream>>>(a); break;
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward_typed(BackwardArgs& a, int num_sms, int* blocks, cudaStream_t stream) {
  constexpr int N = kChunk<T>, e = sizeof(T);
  const bool aligned = a.d % N == 0 && chunk_aligned(a.dy.ptr, a.dy.stride, a.T, e) &&
                       chunk_aligned(a.z.ptr, a.z.stride, a.T, e) &&
                       (!a.dz.ptr || chunk_aligned(a.dz.ptr, a.dz.stride, a.T, e)) &&
                       chunk_aligned(a.dx, a.d, a.T, e) && chunk_aligned(a.w, 0, 1, a.w_f32 ? 4 : e);
  const int chunks = (a.d + N - 1) / N;
  a.tpr = threads_per_row(chunks, 3);
  if (a.tpr > 512) {
    backward_long_kernel<T><<<static_cast<unsigned>(a.T), 1024, 0, stream>>>(a);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess || !(a.want_w || a.want_b)) return err;
    const int slices = static_cast<int>(a.T < 64 ? a.T : 64);
    *blocks = slices;
    column_sums_kernel<T><<<dim3((a.d + 255) / 256, slices), 256, 0, stream>>>(a, slices);
    return cudaGetLastError();
  }
  const int per_thread = (chunks + a.tpr - 1) / a.tpr;
  const int block = a.tpr < 256 ? (a.tpr < 64 ? 128 : a.tpr) : a.tpr;
  const int groups = block / a.tpr;
  const int64_t want = (a.T + groups - 1) / groups;
  const int most = num_sms * (1024 / block) < kNormMaxBlocks ? num_sms * (1024 / block) : kNormMaxBlocks;
  const int grid = static_cast<int>(want < most ? want : most);
  *blocks = grid;
  const size_t smem = groups > 1 ? static_cast<size_t>(a.d) * 4 : 0;
  return aligned ? backward_launch<T, true>(a, per_thread, block, grid, smem, stream)
                 : backward_launch<T, false>(a, per_thread, block, grid, smem, stream);
}

}  // namespace

size_t norm_backward_workspace_bytes(int64_t T, int d) {
  const int64_t blocks = T < kNormMaxBlocks ? T : kNormMaxBlocks;
  return align_up(static_cast<size_t>(blocks < 1 ? 1 : blocks) * 2 * d * 4);
}

cudaError_t launch_layer_norm(const NormForward& f, cudaStream_t stream) {
  ForwardArgs a{{f.x, f.x_stride}, {f.residual, f.residual_stride}, f.weight, f.bias, f.weight_dtype == MOE_F32,
                f.T, f.d, f.eps, f.y, f.z, f.stats, 0, false};
  switch (f.dtype) {
    case MOE_F32: return forward_typed<float>(a, stream);
    case MOE_BF16: return forward_typed<__nv_bfloat16>(a, stream);
    default: return forward_typed<__half>(a, stream);
  }
}

cudaError_t launch_layer_norm_backward(const NormBackward& f, int num_sms, cudaStream_t stream) {
  BackwardArgs a{{f.dy, f.dy_stride}, {f.z, f.z_stride}, {f.dz, f.dz_stride}, f.stats, f.weight,
                 f.weight_dtype == MOE_F32, f.T, f.d, f.dx, f.partial, f.dweight != nullptr, f.dbias != nullptr, 0,
                 false};
  int blocks = 0;
  cudaError_t err;
  switch (f.dtype) {
    case MOE_F32: err = backward_typed<float>(a, num_sms, &blocks, stream); break;
    case MOE_BF16: err = backward_typed<__nv_bfloat16>(a, num_sms, &blocks, stream); break;
    default: err = backward_typed<__half>(a, num_sms, &blocks, stream); break;
  }
  if (err != cudaSuccess || !(a.want_w || a.want_b)) return err;
  finish_kernel<<<dim3((f.d + 31) / 32, 2), 256, 0, stream>>>(f.partial, blocks, f.d, f.dweight, f.dbias);
  return cudaGetLastError();
}

}  // namespace moe
