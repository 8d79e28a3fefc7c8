// Layer norm, backward (the formulas and the forms: layer_norm.cuh).
#pragma once

#include "layer_norm.cuh"

namespace moe {
namespace {

// Rows in flight: what the SM's shared memory holds with three operands, at
// most 432 bytes a thread.
constexpr uint32_t kPitch = kRingThreads * 16;  // bytes between a thread's slots
template <int kChunks>
constexpr int kBackwardStages = kChunks == 1 ? 8 : kChunks == 2 ? 4 : kChunks == 3 ? 3 : 2;

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

// Rows in rings, fixed shares of them for each block (so that a column's sum
// is added in the same order every time), one exchange a row for mean g and
// mean(g n) together.  Bound by memory: 16,384 x 6,144 bf16 with dz 120 us =
// 6.7 TB/s, then the finish kernel; by its instructions for rows that do not
// start on a chunk.
template <typename T, int kChunks, Fit kFit, int kTpr>
__global__ void __launch_bounds__(kRingThreads, 1) backward_ring_kernel(const BackwardArgs a) {
  constexpr int P = kPairs<T>, S = kBackwardStages<kChunks>;
  constexpr bool kKeep = kChunks * P <= 8;  // at most 16 values a thread
  constexpr bool kAligned = kFit != kAnywhere;
  extern __shared__ uint4 ring[];  // [stage][operand][chunk][thread]
  __shared__ float2 red[2][kMaxWarps];
  let_next_start();
  const int tpr = kTpr ? kTpr : a.tpr;
  const int groups = kRingThreads / tpr, lane = threadIdx.x % tpr;
  const bool add = a.dz.ptr != nullptr;
  const uint32_t own = smem_addr(ring) + threadIdx.x * 16, stage_bytes = (add ? 3 : 2) * kChunks * kPitch;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups;
  const int64_t rounds = (a.T - first + step - 1) / step;
  int64_t t = first + threadIdx.x / tpr;
  const Place<T, kChunks, kFit> at(lane, tpr, a.d, kAligned ? 0 : row_offset<T>(a.dy, t));
  const T* dy = static_cast<const T*>(a.dy.ptr) + t * a.dy.stride;
  const T* z = static_cast<const T*>(a.z.ptr) + t * a.z.stride;
  const T* dz = static_cast<const T*>(a.dz.ptr) + (add ? t * a.dz.stride : 0);
  const int64_t out_step = step * a.d;
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
    // Each chunk is behind a check, also where it cannot fail.  Without it the
    // compiler moves all chunks' loads to the front and an SM runs faster by
    // itself, but with a fixed share of the rows for each SM (fixed, so that
    // the column sums are the same every time) all of them together ran
    // slower: 64k x 6144 rows 411 us against 349, 64k x 2048 151 against 129.
    if (live) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (at.j0[c] >= a.d) continue;
        float2 g[P], n[P];
        unpack_pairs<T>(at.load(stage + c * kPitch, c), g);
        unpack_pairs<T>(at.load(stage + (kChunks + c) * kPitch, c), n);
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
    const float2 sum = group_reduce(make_float2(s1.x + s1.y, s2.x + s2.y), tpr, red[round & 1]);
    if (live) {
      const float2 m1 = both(-sum.x * inv_d), c2 = both(-sum.y * inv_d);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        if (at.j0[c] >= a.d) continue;
        float2 g[P], n[P];
        if (kKeep) {
#pragma unroll
          for (int i = 0; i < P; ++i)
            g[i] = fma2(n_row[kKeep ? c * P + i : 0], c2, add2(gw_row[kKeep ? c * P + i : 0], m1));
        } else {
          unpack_pairs<T>(at.load(stage + c * kPitch, c), g);
          unpack_pairs<T>(at.load(stage + (kChunks + c) * kPitch, c), n);
#pragma unroll
          for (int i = 0; i < P; ++i)
            g[i] = fma2(mul2(add2(n[i], m2), r2), c2, fma2(g[i], w[c * P + i], m1));
        }
        if (add) {
          unpack_pairs<T>(at.load(stage + (2 * kChunks + c) * kPitch, c), n);
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
    dx += out_step;
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

// Operands whose rows lie differently within 16 bytes: single values, the
// column sums in registers.  Bound by the latency of narrow loads; fixed
// shares as above.
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

// Rows too long for the registers: dx by a block a row, which keeps dy and z
// in shared memory between its two sweeps (`cached`, else they are read
// again), and the column sums by a block for each run of columns and slice of
// rows, whose lanes read neighbouring columns: dy and z are read twice in all,
// which a row of this length leaves no registers to avoid (8,192 x 32,768 bf16:
// 685 us, with dz 732, where reading once would take 237 and 316).
template <typename T, bool kVec>
__global__ void __launch_bounds__(1024) backward_long_kernel(const BackwardArgs a, bool cached) {
  using U = Unit<T, kVec>;
  using Store = typename U::Store;
  extern __shared__ uint4 row_cache[];
  __shared__ float2 red[kMaxWarps];
  const int64_t t = blockIdx.x;
  const int units = a.d / U::N;
  const Store* dy = reinterpret_cast<const Store*>(static_cast<const T*>(a.dy.ptr) + t * a.dy.stride);
  const Store* z = reinterpret_cast<const Store*>(static_cast<const T*>(a.z.ptr) + t * a.z.stride);
  const Store* dz = reinterpret_cast<const Store*>(static_cast<const T*>(a.dz.ptr) + (a.dz.ptr ? t * a.dz.stride : 0));
  Store* dx = reinterpret_cast<Store*>(static_cast<T*>(a.dx) + t * a.d);
  Store* cache = reinterpret_cast<Store*>(row_cache);
  const float mu = a.stats[t], r = a.stats[a.T + t];
  float g[U::N], n[U::N], p[U::N];
  float2 s = make_float2(0.0f, 0.0f);
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    const Store raw_g = dy[u], raw_n = z[u];
    if (cached) cache[u] = raw_g, cache[units + u] = raw_n;
    U::values(raw_g, g);
    U::values(raw_n, n);
    U::params(a.w, a.w_f32, 1.0f, u, p);
#pragma unroll
    for (int i = 0; i < U::N; ++i) {
      s.x += g[i] * p[i];
      s.y += g[i] * p[i] * ((n[i] - mu) * r);
    }
  }
  // each thread reads back only what it has written itself
  const Store* dy_in = cached ? cache : dy;
  const Store* z_in = cached ? cache + units : z;
  s = group_reduce(s, blockDim.x, red);
  s.x /= static_cast<float>(a.d);
  s.y /= static_cast<float>(a.d);
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    U::values(dy_in[u], g);
    U::values(z_in[u], n);
    U::params(a.w, a.w_f32, 1.0f, u, p);
#pragma unroll
    for (int i = 0; i < U::N; ++i) g[i] = (g[i] * p[i] - s.x - (n[i] - mu) * r * s.y) * r;
    if (a.dz.ptr) {
      U::values(dz[u], p);
#pragma unroll
      for (int i = 0; i < U::N; ++i) g[i] += p[i];
    }
    dx[u] = U::store(g);
  }
}

constexpr int kColumnThreads = 128;
template <typename T, bool kVec>
__global__ void __launch_bounds__(kColumnThreads) column_sums_kernel(const BackwardArgs a, int slices) {
  using U = Unit<T, kVec>;
  using Store = typename U::Store;
  let_next_start();
  const int u = blockIdx.x * kColumnThreads + threadIdx.x;
  if (u >= a.d / U::N) return;
  float sw[U::N], sb[U::N], g[U::N], n[U::N];
#pragma unroll
  for (int i = 0; i < U::N; ++i) sw[i] = sb[i] = 0.0f;
#pragma unroll 4
  for (int64_t t = blockIdx.y; t < a.T; t += slices) {
    U::values(reinterpret_cast<const Store*>(static_cast<const T*>(a.dy.ptr) + t * a.dy.stride)[u], g);
    U::values(reinterpret_cast<const Store*>(static_cast<const T*>(a.z.ptr) + t * a.z.stride)[u], n);
    const float mu = __ldg(a.stats + t), r = __ldg(a.stats + a.T + t);
#pragma unroll
    for (int i = 0; i < U::N; ++i) {
      sw[i] += g[i] * ((n[i] - mu) * r);
      sb[i] += g[i];
    }
  }
  float* out = a.partial + static_cast<int64_t>(blockIdx.y) * 2 * a.d + u * U::N;
#pragma unroll
  for (int i = 0; i < U::N; ++i) {
    if (a.want_w) out[i] = sw[i];
    if (a.want_b) out[a.d + i] = sb[i];
  }
}

// ---- host
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

template <typename T, int kChunks, Fit kFit, int kTpr>
cudaError_t backward_ring(BackwardArgs& a, int num_sms, int* blocks, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr bool kAligned = kFit != kAnywhere;
  constexpr size_t operand = static_cast<size_t>(kBackwardStages<kChunks>) * kChunks * kPitch;
  auto kernel = backward_ring_kernel<T, kChunks, kFit, kTpr>;
  const cudaError_t err = allow(reinterpret_cast<const void*>(kernel), done, 3 * operand, true);
  if (err != cudaSuccess) return err;
  const size_t smem = (a.dz.ptr ? 3 : 2) * operand;
  const int groups = kRingThreads / a.tpr;
  const int multiple = kAligned || groups >= kChunk<T> ? 1 : kChunk<T> / groups;
  a.cluster = cluster_blocks(a.T, groups, multiple);
  if (a.cluster) return launch_cluster(kernel, a.cluster, kRingThreads, smem, stream, a);
  *blocks = ring_grid(a.T, groups, kChunk<T>, kAligned, num_sms);
  kernel<<<*blocks, kRingThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

// The kernel made for this number of threads.
template <typename T, int kChunks, Fit kFit>
cudaError_t backward_sized(BackwardArgs& a, int num_sms, int* blocks, cudaStream_t stream) {
  if constexpr (kChunks == 4) {
    return backward_ring<T, kChunks, kFit, 512>(a, num_sms, blocks, stream);
  } else if constexpr (kChunks > 1) {
    switch (a.tpr) {
      case 32: return backward_ring<T, kChunks, kFit, 32>(a, num_sms, blocks, stream);
      case 64: return backward_ring<T, kChunks, kFit, 64>(a, num_sms, blocks, stream);
      case 128: return backward_ring<T, kChunks, kFit, 128>(a, num_sms, blocks, stream);
      case 256: return backward_ring<T, kChunks, kFit, 256>(a, num_sms, blocks, stream);
      default: return backward_ring<T, kChunks, kFit, 512>(a, num_sms, blocks, stream);
    }
  } else {
    return backward_ring<T, kChunks, kFit, 0>(a, num_sms, blocks, stream);
  }
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

template <typename T, bool kVec>
cudaError_t backward_long(const BackwardArgs& a, int* blocks, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto kernel = backward_long_kernel<T, kVec>;
  cudaError_t err = allow(reinterpret_cast<const void*>(kernel), done, kLongCache, false);
  if (err != cudaSuccess) return err;
  const size_t bytes = static_cast<size_t>(a.d) * sizeof(T) * 2;
  const bool cached = bytes <= kLongCache;
  kernel<<<static_cast<unsigned>(a.T), 1024, cached ? bytes : 0, stream>>>(a, cached);
  err = cudaGetLastError();
  if (err != cudaSuccess || !(a.want_w || a.want_b)) return err;
  *blocks = static_cast<int>(a.T < 64 ? a.T : 64);
  const int units = a.d / Unit<T, kVec>::N;
  column_sums_kernel<T, kVec>
      <<<dim3((units + kColumnThreads - 1) / kColumnThreads, *blocks), kColumnThreads, 0, stream>>>(a, *blocks);
  return cudaGetLastError();
}

template <typename T, Fit kFit>
cudaError_t backward_fit(BackwardArgs& a, int per_thread, int num_sms, int* blocks, cudaStream_t stream) {
  if (per_thread == 1) return backward_sized<T, 1, kFit>(a, num_sms, blocks, stream);
  if (per_thread == 2) return backward_sized<T, 2, kFit>(a, num_sms, blocks, stream);
  if (per_thread == 3) return backward_sized<T, 3, kFit>(a, num_sms, blocks, stream);
  return backward_sized<T, 4, kFit>(a, num_sms, blocks, stream);
}

}  // namespace

template <typename T>
cudaError_t norm_backward_typed(BackwardArgs& a, int num_sms, int* blocks, cudaStream_t stream) {
  constexpr int N = kChunk<T>, e = sizeof(T);
  Lie lie(a.dy.ptr, a.T > 1 ? a.dy.stride * e : a.d * e);
  lie.add(a.z.ptr, a.T > 1 ? a.z.stride * e : a.d * e);
  if (a.dz.ptr) lie.add(a.dz.ptr, a.T > 1 ? a.dz.stride * e : a.d * e);
  lie.add(a.dx, static_cast<int64_t>(a.d) * e);
  const bool aligned = lie.on_chunks && a.d % N == 0 && param_on_chunks(a.w);
  int per_thread = 0;
  if (aligned || lie.alike) a.tpr = ring_threads(a.d, N, aligned, &per_thread);
  if (a.tpr > 0) {
    const Fit fit = !aligned ? kAnywhere : a.d == a.tpr * per_thread * N ? kFull : kOnChunks;
    if (fit == kFull) return backward_fit<T, kFull>(a, per_thread, num_sms, blocks, stream);
    return fit == kOnChunks ? backward_fit<T, kOnChunks>(a, per_thread, num_sms, blocks, stream)
                            : backward_fit<T, kAnywhere>(a, per_thread, num_sms, blocks, stream);
  }
  a.tpr = threads_per_row(a.d, a.d <= 2048 ? 8 : 16);
  if (a.tpr <= kRingThreads) {
    const int values = (a.d + a.tpr - 1) / a.tpr;
    if (values <= 4) return backward_values<T, 4>(a, num_sms, blocks, stream);
    if (values <= 8) return backward_values<T, 8>(a, num_sms, blocks, stream);
    return backward_values<T, 16>(a, num_sms, blocks, stream);
  }
  return aligned ? backward_long<T, true>(a, blocks, stream) : backward_long<T, false>(a, blocks, stream);
}

}  // namespace moe
