// Layer norm, forward (the formulas and the forms: layer_norm.cuh).
#pragma once

#include "layer_norm.cuh"

namespace moe {
namespace {

// A group of kOwnBlock threads or more is a block of its own.
constexpr int kOwnBlock = 64, kSmallBlock = 128;
// A group works on kBatch rows at a time (a round), so that the reductions of
// one row run beside those of another; the rounds in flight are what an SM's
// shared memory holds for 512 threads with two operands.
template <int kChunks>
constexpr int kBatch = kChunks <= 2 ? 2 : 1;
template <int kChunks>
constexpr int kForwardStages = kChunks == 1 ? 6 : kChunks == 3 ? 4 : 3;

// A block's piece: `tile_rounds` rounds of kBatch rows a group.  On chunks, the
// pieces are runs of consecutive rows, one for each launched block, and
// blocks steal the launches that still wait: the SMs are not equally near to
// all of the memory, and an equal share for each took 10 % longer (64k x 6144
// rows with a residual: 537 us, with 4 blocks an SM 488 us).  Rows that do
// not start on a chunk are dealt out round by round, so that a group's rows
// start alike.
//
// kTpr: the threads of a row where that is known when compiling, or 0.  A
// group of kOwnBlock threads or more is a block of its own (blocks meet at
// every piece).
//
// Bound by memory: 64k x 6144 bf16 with a residual 466 us = 6.9 TB/s, 64k x
// 2048 without 81 us = 6.6 TB/s.  Rows that do not start on a chunk keep
// fixed shares and checks of their ends, and are bound by their instructions:
// 34,462 x 3,570 fp16 with a residual 216 us = 4.6 TB/s.  The reciprocal root
// is the approximate one, right to two units in the last place of fp32, which
// the variance's own sum leaves too.
template <typename T, int kChunks, Fit kFit, int kTpr>
__global__ void __launch_bounds__(kRingThreads, 1) forward_ring_kernel(const ForwardArgs a) {
  constexpr int P = kPairs<T>, S = kForwardStages<kChunks>, B = kBatch<kChunks>;
  constexpr bool kAligned = kFit != kAnywhere;
  extern __shared__ uint4 ring[];  // [stage][row][operand][chunk][thread]
  const int tpr = kTpr ? kTpr : a.tpr;
  __shared__ float2 red[2][B * kMaxWarps];
  __shared__ uint4 answer;
  __shared__ uint64_t answer_bar;
  constexpr bool kOneGroup = kTpr >= kOwnBlock;  // the block is the group
  const int groups = kOneGroup ? 1 : (kTpr ? kSmallBlock : blockDim.x) / tpr;
  const int lane = kOneGroup ? threadIdx.x : threadIdx.x % tpr, group = kOneGroup ? 0 : threadIdx.x / tpr;
  const bool res = a.res.ptr != nullptr;
  // bytes between a thread's slots: those of a chunk of the whole block
  const uint32_t pitch = (kOneGroup ? kTpr : kTpr ? kSmallBlock : blockDim.x) * 16;
  const uint32_t row_bytes = (res ? 2 : 1) * kChunks * pitch, stage_bytes = B * row_bytes;
  const uint32_t own = smem_addr(ring) + threadIdx.x * 16;
  const int64_t step = kAligned ? groups : static_cast<int64_t>(gridDim.x) * groups;
  const int64_t first = blockIdx.x * a.piece + group;
  const int64_t end = kAligned && !a.steal ? min(a.T, (blockIdx.x + 1) * a.piece) : a.T;
  if (kAligned && a.steal && threadIdx.x == 0) {
    mbar_init(&answer_bar, 1);
    fence_barrier_init();
    steal_request(&answer, &answer_bar);
  }
  const Place<T, kChunks, kFit> at(lane, tpr, a.d, kAligned ? 0 : row_offset<T>(a.x, first));
  // the row that is fetched next, its round in the piece, and the block's
  // first row in the piece after the one being worked on (T: there is none)
  int64_t ahead = first, next_piece = a.T;
  int ahead_round = 0;
  uint32_t answers = 0;
  const T* x = static_cast<const T*>(a.x.ptr) + first * a.x.stride;
  const T* r_row = static_cast<const T*>(a.res.ptr) + (res ? first * a.res.stride : 0);
  auto fetch = [&](uint32_t stage) {
#pragma unroll
    for (int k = 0; k < B; ++k, stage += row_bytes) {
      if (ahead < end) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (!at.any(c)) continue;
          at.fetch(stage + c * pitch, x, c);
          if (res) at.fetch(stage + (kChunks + c) * pitch, r_row, c);
        }
      }
      ahead += step;
      x += step * a.x.stride;
      if (res) r_row += step * a.res.stride;
    }
    copy_commit();
  };
  // Moves on to the next piece after the last round of one.  Every thread of
  // the block comes here in the same round.
  auto advance = [&]() {
    if (!kAligned || ++ahead_round < a.tile_rounds) return;
    ahead_round = 0;
    next_piece = ahead = a.T;
    if (!a.steal || answers >= kStealLost) return;
    if (answers == 0) __syncthreads();  // the barrier is initialised
    const int block = steal_next(&answer, &answer_bar, answers & 1);
    answers = block >= 0 ? answers + 1 : block == kStealRefused ? kStealOver : kStealLost;
    if (block < 0) return;
    if (threadIdx.x == 0) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      steal_request(&answer, &answer_bar);
    }
    next_piece = block * a.piece;
    ahead = next_piece + group;
    x = static_cast<const T*>(a.x.ptr) + ahead * a.x.stride;
    if (res) r_row = static_cast<const T*>(a.res.ptr) + ahead * a.res.stride;
  };
  for (int s = 0; s < S - 1; ++s) {
    fetch(own + s * stage_bytes);
    advance();
  }
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
  const float n_warp = warp_reduce(static_cast<float>(count), tpr);
  const float inv_n = n_warp > 0.0f ? 1.0f / n_warp : 0.0f;
  float n_other = 0.0f, inv_other = 0.0f;  // of the warp that exchange() hands over
  if (tpr > 32) {
    const float2 other = exchange(make_float2(n_warp, inv_n), tpr, group, red[1]);
    n_other = other.x, inv_other = other.y;
  }
  uint32_t stage = own, next = own + (S - 1) * stage_bytes;
  int64_t t = first;
  int round = 0;
  const int64_t out_step = step * a.d;
  T* y = static_cast<T*>(a.y) + t * a.d;
  T* z = static_cast<T*>(a.z) + (res ? t * a.d : 0);
  // Rows beyond the end are worked on like others, on whatever their slots
  // hold, and not written: no branch parts the rows of a round.
  for (uint32_t parity = 0;; parity ^= 1) {
    fetch(next);
    advance();
    copy_wait<S - 1>();
    float2 v[B][kChunks * P], sq[B];
    float mid[B], mu[B], r[B];
    bool live[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      live[k] = t + k * step < end;
      float2 s = both(0.0f);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint4 u = at.load(stage + k * row_bytes + c * pitch, c);
        if (res) {
          // the sum is rounded to the rows' type here: it is what the caller
          // keeps and what the backward normalises again
          u = add_chunks<T>(u, at.load(stage + k * row_bytes + (kChunks + c) * pitch, c));
          if (live[k] && at.any(c)) at.store(z + k * out_step, c, u);
        }
        unpack_pairs<T>(u, v[k] + c * P);
        at.mask(c, v[k] + c * P, 0.0f);
#pragma unroll
        for (int i = 0; i < P; ++i) s = add2(s, v[k][c * P + i]);
      }
      sq[k].x = s.x + s.y;
    }
#pragma unroll
    for (int k = 0; k < B; ++k) {
      sq[k].x = warp_reduce(sq[k].x, tpr);
      mid[k] = sq[k].x * inv_n;  // the warp's mean
    }
#pragma unroll
    for (int k = 0; k < B; ++k) {
      float2 s = both(0.0f);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        at.mask(c, v[k] + c * P, mid[k]);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          float2& e = v[k][c * P + i];
          e = add2(e, both(-mid[k]));
          s = fma2(e, e, s);
        }
      }
      sq[k].y = s.x + s.y;
    }
#pragma unroll
    for (int k = 0; k < B; ++k) {
      sq[k].y = warp_reduce(sq[k].y, tpr);
      mu[k] = mid[k];
    }
    if (tpr > 32) {
      exchange(sq, tpr, group, red[parity]);
#pragma unroll
      for (int k = 0; k < B; ++k) {
        mu[k] = over_warps(sq[k].x, tpr >> 5) * inv_d;
        const float e = sq[k].x * inv_other - mu[k];
        sq[k].y = over_warps(fmaf(n_other * e, e, sq[k].y), tpr >> 5);
      }
    }
#pragma unroll
    for (int k = 0; k < B; ++k) r[k] = rsqrtf(fmaf(sq[k].y, inv_d, a.eps));
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < B; ++k) {
        if (!live[k]) continue;
        a.stats[t + k * step] = mu[k];
        a.stats[a.T + t + k * step] = r[k];
      }
    }
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const float2 r2 = both(r[k]), shift = both((mid[k] - mu[k]) * r[k]);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        // (z - mu) r = (z - mid) r + (mid - mu) r
#pragma unroll
        for (int i = 0; i < P; ++i) {
          float2& e = v[k][c * P + i];
          e = fma2(fma2(e, r2, shift), w[c * P + i], b[c * P + i]);
        }
        if (live[k] && at.any(c)) at.store(y + k * out_step, c, pack_pairs<T>(v[k] + c * P));
      }
    }
    next = stage;
    stage = stage + stage_bytes == own + S * stage_bytes ? own : stage + stage_bytes;
    t += B * step;
    y += B * out_step;
    if (res) z += B * out_step;
    if (++round < a.tile_rounds) continue;
    if (next_piece >= a.T) {
      // a piece may be lost: NaN in the first row of this one (which this
      // thread wrote) says so
      if (answers == kStealLost && threadIdx.x == 0) {
        const int64_t row = t - a.piece;
        a.stats[row] = a.stats[a.T + row] = nanf("");
        static_cast<T*>(a.y)[row * a.d] = from_f32<T>(nanf(""));
      }
      return;
    }
    round = 0;
    t = next_piece + group;
    y = static_cast<T*>(a.y) + t * a.d;
    if (res) z = static_cast<T*>(a.z) + t * a.d;
  }
}

// Operands whose rows lie differently within 16 bytes, single values in
// registers: bound by the latency of narrow loads, which a row's one batch of
// them has to cover, so every group takes one row and the SM holds as many
// groups as fit.
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

// Rows beyond the rings, one block a row in three sweeps (mean, deviations,
// output): bound by the two exchanges a row, between which a block reads
// nothing (8,192 x 32,768 bf16: 299 us = 3.6 TB/s, with a residual 395 us = 5.4
// TB/s), and where a row's start allows single values only (kVec false) by its
// instructions (4,000 x 15,001 fp32: 231 us = 2.1 TB/s).  `cached`: the
// row stays in shared memory between sweeps, else they read it again.
template <typename T, bool kVec>
__global__ void __launch_bounds__(1024) forward_long_kernel(const ForwardArgs a, bool cached) {
  using U = Unit<T, kVec>;
  using Store = typename U::Store;
  extern __shared__ uint4 row_cache[];
  __shared__ float2 red[2][kMaxWarps];
  const int64_t t = blockIdx.x;
  const int units = a.d / U::N;
  const Store* x = reinterpret_cast<const Store*>(static_cast<const T*>(a.x.ptr) + t * a.x.stride);
  const Store* res =
      reinterpret_cast<const Store*>(static_cast<const T*>(a.res.ptr) + (a.res.ptr ? t * a.res.stride : 0));
  Store* z = reinterpret_cast<Store*>(static_cast<T*>(a.z) + (a.res.ptr ? t * a.d : 0));
  Store* y = reinterpret_cast<Store*>(static_cast<T*>(a.y) + t * a.d);
  Store* cache = reinterpret_cast<Store*>(row_cache);
  float v[U::N], p[U::N];
  float s = 0.0f;
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    Store raw = x[u];
    U::values(raw, v);
    if (a.res.ptr) {
      U::values(res[u], p);
#pragma unroll
      for (int i = 0; i < U::N; ++i) v[i] += p[i];
      raw = U::store(v);
      z[u] = raw;
      U::values(raw, v);
    }
    if (cached) cache[u] = raw;
#pragma unroll
    for (int i = 0; i < U::N; ++i) s += v[i];
  }
  // each thread reads back only what it has written itself
  const Store* in = cached ? cache : a.res.ptr ? z : x;
  const float mu = group_reduce(s, blockDim.x, red[0]) / static_cast<float>(a.d);
  s = 0.0f;
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    U::values(in[u], v);
#pragma unroll
    for (int i = 0; i < U::N; ++i) s += (v[i] - mu) * (v[i] - mu);
  }
  const float r = rsqrtf(group_reduce(s, blockDim.x, red[1]) / static_cast<float>(a.d) + a.eps);
  if (threadIdx.x == 0) {
    a.stats[t] = mu;
    a.stats[a.T + t] = r;
  }
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    U::values(in[u], v);
    U::params(a.w, a.w_f32, 1.0f, u, p);
#pragma unroll
    for (int i = 0; i < U::N; ++i) v[i] = (v[i] - mu) * r * p[i];
    U::params(a.b, a.w_f32, 0.0f, u, p);
#pragma unroll
    for (int i = 0; i < U::N; ++i) v[i] += p[i];
    y[u] = U::store(v);
  }
}

// ---- host
// Rounds of a stolen piece: no fewer than the rounds in flight, so that only
// one piece is ahead of the one being worked on; few, so that the SMs end
// together.
template <int kChunks>
constexpr int kStealRounds = kForwardStages<kChunks> > 4 ? kForwardStages<kChunks> : 4;

template <typename T, int kChunks, Fit kFit, int kTpr>
cudaError_t forward_ring(ForwardArgs& a, int num_sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr bool kAligned = kFit != kAnywhere;
  constexpr int B = kBatch<kChunks>;
  constexpr uint32_t used = kForwardStages<kChunks> * B * kChunks;
  // groups of 64 threads as blocks of their own only where that is known when
  // compiling (4095 x 1001 bf16: 16.5 us against 10.1 in blocks of 128)
  const int block = a.tpr < (kTpr ? kOwnBlock : kSmallBlock) ? kSmallBlock : a.tpr, groups = block / a.tpr;
  auto kernel = forward_ring_kernel<T, kChunks, kFit, kTpr>;
  const cudaError_t err = allow(reinterpret_cast<const void*>(kernel), done,
                                static_cast<size_t>(2 * used) * 16 * kRingThreads, false);
  if (err != cudaSuccess) return err;
  int grid = ring_grid(a.T, groups, kChunk<T>, kAligned, num_sms * (kRingThreads / block));
  const int64_t per_round = static_cast<int64_t>(grid) * groups * B;
  a.tile_rounds = static_cast<int>((a.T + per_round - 1) / per_round);
  a.piece = groups;
  a.steal = kAligned && a.tile_rounds >= 2 * kStealRounds<kChunks>;
  if (kAligned) {
    if (a.steal) a.tile_rounds = kStealRounds<kChunks>;
    // rows enough for one round or less are spread over the blocks first
    const int64_t once = static_cast<int64_t>(grid) * groups;
    a.piece = a.tile_rounds == 1 ? (a.T + once - 1) / once * groups : static_cast<int64_t>(a.tile_rounds) * B * groups;
    grid = static_cast<int>((a.T + a.piece - 1) / a.piece);
  }
  const size_t smem = static_cast<size_t>(used) * (a.res.ptr ? 2 : 1) * 16 * block;
  kernel<<<grid, block, smem, stream>>>(a);
  return cudaGetLastError();
}

// The kernel made for this number of threads, where rows start on chunks.
template <typename T, int kChunks, Fit kFit>
cudaError_t forward_sized(ForwardArgs& a, int num_sms, cudaStream_t stream) {
  if constexpr (kChunks > 1 && kFit != kAnywhere) {
    switch (a.tpr) {
      case 32: return forward_ring<T, kChunks, kFit, 32>(a, num_sms, stream);
      case 64: return forward_ring<T, kChunks, kFit, 64>(a, num_sms, stream);
      case 128: return forward_ring<T, kChunks, kFit, 128>(a, num_sms, stream);
      case 256: return forward_ring<T, kChunks, kFit, 256>(a, num_sms, stream);
      default: return forward_ring<T, kChunks, kFit, 512>(a, num_sms, stream);
    }
  } else {
    return forward_ring<T, kChunks, kFit, 0>(a, num_sms, stream);
  }
}

template <typename T, int kValues>
cudaError_t forward_values(const ForwardArgs& a, cudaStream_t stream) {
  const int block = a.tpr < 128 ? 128 : a.tpr, groups = block / a.tpr;
  forward_values_kernel<T, kValues><<<static_cast<unsigned>((a.T + groups - 1) / groups), block, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, bool kVec>
cudaError_t forward_long(const ForwardArgs& a, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto kernel = forward_long_kernel<T, kVec>;
  const cudaError_t err = allow(reinterpret_cast<const void*>(kernel), done, kLongCache, false);
  if (err != cudaSuccess) return err;
  const size_t bytes = static_cast<size_t>(a.d) * sizeof(T);
  const bool cached = bytes <= kLongCache;
  kernel<<<static_cast<unsigned>(a.T), 1024, cached ? bytes : 0, stream>>>(a, cached);
  return cudaGetLastError();
}

template <typename T, Fit kFit>
cudaError_t forward_fit(ForwardArgs& a, int per_thread, int num_sms, cudaStream_t stream) {
  if (per_thread == 1) return forward_sized<T, 1, kFit>(a, num_sms, stream);
  if (per_thread == 2) return forward_sized<T, 2, kFit>(a, num_sms, stream);
  if (per_thread == 3) return forward_sized<T, 3, kFit>(a, num_sms, stream);
  if constexpr (kFit == kAnywhere) return forward_ring<T, 4, kFit, 0>(a, num_sms, stream);
  else if (a.tpr == 32) return forward_ring<T, 4, kFit, 32>(a, num_sms, stream);
  else return forward_ring<T, 4, kFit, 512>(a, num_sms, stream);
}

}  // namespace

template <typename T>
cudaError_t norm_forward_typed(ForwardArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int N = kChunk<T>, e = sizeof(T);
  Lie lie(a.x.ptr, a.T > 1 ? a.x.stride * e : a.d * e);
  lie.add(a.y, static_cast<int64_t>(a.d) * e);
  if (a.res.ptr) {
    lie.add(a.res.ptr, a.T > 1 ? a.res.stride * e : a.d * e);
    lie.add(a.z, static_cast<int64_t>(a.d) * e);
  }
  const bool aligned = lie.on_chunks && a.d % N == 0 && param_on_chunks(a.w) && param_on_chunks(a.b);
  const int chunks = (a.d + N - 1) / N;
  int per_thread = 0;
  if (aligned || lie.alike) a.tpr = ring_threads(a.d, N, aligned, &per_thread);
  // up to 4 chunks a thread where that keeps a row inside a warp: no barrier
  // (64k x 1024 bf16: 43 us against 56 with 2 chunks and 64 threads)
  if (aligned && a.tpr == 64 && chunks <= 128) a.tpr = 32, per_thread = 4;
  if (a.tpr > 0) {
    const Fit fit = !aligned ? kAnywhere : a.d == a.tpr * per_thread * N ? kFull : kOnChunks;
    if (fit == kFull) return forward_fit<T, kFull>(a, per_thread, num_sms, stream);
    return fit == kOnChunks ? forward_fit<T, kOnChunks>(a, per_thread, num_sms, stream)
                            : forward_fit<T, kAnywhere>(a, per_thread, num_sms, stream);
  }
  // at most 8 values a thread: more spill at 1,024 threads
  a.tpr = threads_per_row(a.d, 8);
  if (a.tpr <= 1024)
    return a.d <= a.tpr * 4 ? forward_values<T, 4>(a, stream) : forward_values<T, 8>(a, stream);
  return aligned ? forward_long<T, true>(a, stream) : forward_long<T, false>(a, stream);
}

}  // namespace moe
