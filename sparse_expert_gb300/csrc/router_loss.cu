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
// The rows are cut into pieces of a few rounds, one for each launched block,
// and running blocks steal the launches that still wait; each piece leaves
// its own sums, which are added in the pieces' order, so it does not matter
// which block did it.
//
// The mask is counted by a kernel of its own first: every block needs N, and
// where each counted for itself that cost more than the losses (65,536
// tokens: 349 us in all).  A small problem is one cluster of blocks that
// count, and add up the losses, among themselves: one launch.
//
// Bound by latency: a row's maximum and its two sums are ten exchanges that
// wait on one another, and 20 warps an SM do not cover them.  65,536 x 384
// added to a gradient, with or without a mask: 58 us, of which this kernel 47
// (25 instructions a value in 39 % of the issue slots, 64 % of the device's
// memory rate) and reading and writing alone 44.5; the rest is the count before
// and the last sums behind.  Written fresh: 42-46 us against 30.  30,000 rows
// of 768 and 1,000, added: 58 and 75 us against 41 and 53.
#include "common.cuh"
#include "elem.cuh"
#include "internal.h"
#include "launch.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kCountBlocks = 64;

struct Args {
  RouterLoss a;
  const int32_t* kept;  // [kCountBlocks] tokens kept, by the counting kernel; null without a mask
  float2* partial;      // [pieces]: sums of s_t and lse_t^2, unless one cluster adds them up
  int tpr;
  int cluster;          // its blocks, or 0
  int rounds;           // of a piece
  bool steal;
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

// Two sums over a group's lanes, their exchanges side by side.
__device__ __forceinline__ float2 group_sums(float2 v, int width) {
  if (width == 32) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
      v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, s), __shfl_xor_sync(0xffffffffu, v.y, s)));
  } else {
    for (int s = width >> 1; s > 0; s >>= 1)
      v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, s), __shfl_xor_sync(0xffffffffu, v.y, s)));
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

// 2^v for -126 <= v (0 below).  Approximate, as are the quotient and the
// logarithm of a row's sum below: a few units in the last place of fp32, as
// much as the sum itself leaves.
__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Rows in flight a group: this one and the next.  Blocks an SM: the registers
// of a lane's values, and no more, bound them (65,536 x 384, 12 values a lane:
// 5 blocks 56.6 us, 6 blocks 57.8, 7 blocks 60.7; 30,000 x 1,000, 32 values: 3
// blocks 75.3 us, 4 blocks 84.5).
constexpr int kStages = 2;
constexpr int blocks_per_sm(int values) { return values <= 12 ? 5 : values <= 16 ? 4 : 3; }
// Rounds of a stolen piece: no fewer than the rows in flight, so that only one
// piece is ahead; few, so that the SMs end together (30,000 x 1,000: 8 rounds
// 98.6 us, 4 rounds 87.1).
constexpr int kStealRounds = 4;

// kTpr: the lanes of a row where that is known when compiling, or 0.
template <int kValues, bool kVec, bool kFull, int kTpr>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(kValues)) loss_kernel(const Args args) {
  const RouterLoss& a = args.a;
  constexpr int kPairsRow = kValues / 2, S = kStages, kWarps = kThreads / 32;
  constexpr uint32_t kOperand = kValues / (kVec ? 4 : 1) * kPitch<kVec>;
  const int tpr = kTpr ? kTpr : args.tpr, E = kFull && kTpr ? kValues * kTpr : a.E;
  extern __shared__ uint4 ring[];  // [stage][operand][vector or value][thread]
  __shared__ int64_t red_i[kWarps];
  __shared__ float2 red[2][kWarps], block_losses;
  __shared__ uint4 answer;
  __shared__ uint64_t answer_bar;
  let_next_start();
  const int lane = threadIdx.x % tpr, group = threadIdx.x / tpr, groups = kThreads / tpr;
  if (args.steal && threadIdx.x == 0) {
    mbar_init(&answer_bar, 1);
    fence_barrier_init();
    steal_request(&answer, &answer_bar);
  }
  // a piece: args.rounds rounds of a row a group, consecutive rows
  const int64_t piece_rows = static_cast<int64_t>(args.rounds) * groups;
  auto kept_row = [&](int64_t row) { return row < a.T && (!a.mask || __ldg(a.mask + row) != 0); };
  // a masked row of a gradient accumulated in place is left as it is
  const bool in_place = a.d_in && a.d_in == a.d_logits;
  const uint32_t own = smem_addr(ring) + threadIdx.x * (kVec ? 16 : 4), stage_bytes = (a.d_in ? 2 : 1) * kOperand;
  int64_t piece = blockIdx.x, next_piece = -1;
  int64_t ahead = piece * piece_rows + group;
  int ahead_round = 0;
  uint32_t answers = 0;
  bool ahead_live = kept_row(ahead);
  uint32_t live_bits = 0;  // bit k: the row k rounds after this one is kept
  auto fetch = [&](uint32_t stage, int round) {
    if (ahead_live) fetch_row<kValues, kVec, kFull>(stage, a.logits + ahead * E, E, lane, tpr);
    if (a.d_in && ahead < a.T && (ahead_live || !in_place))
      fetch_row<kValues, kVec, kFull>(stage + kOperand, a.d_in + ahead * E, E, lane, tpr);
    asm volatile("cp.async.commit_group;" ::: "memory");
    live_bits |= static_cast<uint32_t>(ahead_live) << round;
    ahead += groups;
    // after a piece's last round, on to the next piece; every thread of the
    // block comes here in the same round
    if (++ahead_round == args.rounds) {
      ahead_round = 0;
      next_piece = -1;
      ahead = a.T;
      if (args.steal && answers < kStealLost) {
        if (answers == 0) __syncthreads();  // the barrier is initialised
        const int block = steal_next(&answer, &answer_bar, answers & 1);
        answers = block >= 0 ? answers + 1 : block == kStealRefused ? kStealOver : kStealLost;
        if (block >= 0) {
          if (threadIdx.x == 0) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            steal_request(&answer, &answer_bar);
          }
          next_piece = block;
          ahead = next_piece * piece_rows + group;
        }
      }
    }
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
  float2 sums = both(0.0f);  // of s_t and lse_t^2 over the piece
  uint32_t stage = own, next = own + (S - 1) * stage_bytes, parity = 0;
  int64_t t = piece * piece_rows + group;
  for (int round = 0;; t += groups, live_bits >>= 1) {
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
    const float2 row_sums = group_sums(make_float2(z2.x + z2.y, dot2.x + dot2.y), tpr);
    const float z = row_sums.x, dot = row_sums.y;
    const bool empty = z == 0.0f;
    const float inv_z = empty ? 0.0f : __fdividef(1.0f, z);  // z in [1, E]
    const float s = dot * inv_z;
    const float lse = empty ? 0.0f : top + __logf(z);
    sums = add2(sums, make_float2(s, lse * lse));
    // p / N (cb (share - s) + cz lse) = e (scale_b share + scale_0)
    const float scale = inv_z * inv_n;
    const float2 scale_b = both(scale * cb), scale_0 = both(scale * (cz * lse - cb * s));
    float* out = a.d_logits + t * E;
#pragma unroll
    for (int i = 0; i < kPairsRow; ++i) {
      l[i] = mul2(l[i], fma2(scale_b, share[i], scale_0));
      if (a.d_in) l[i] = add2(l[i], before[i]);
    }
    if (write) {
#pragma unroll
      for (int i = 0; i < kValues; i += kVec ? 4 : 2) {
        const int e = column<kVec>(i, lane, tpr);
        const float2 lo = l[i / 2];
        if (kVec) {
          const float2 hi = l[i / 2 + (kVec ? 1 : 0)];
          if (kFull || e < E) __stcs(reinterpret_cast<float4*>(out + e), make_float4(lo.x, lo.y, hi.x, hi.y));
        } else {
          if (e < E) out[e] = lo.x;
          if (e + tpr < E) out[e + tpr] = lo.y;
        }
      }
    }
    if (++round < args.rounds) continue;
    // the piece's sums: every lane of a group carries its rows', so the
    // groups of a warp add up, and then the warps
    for (int s = tpr; s < 32; s <<= 1) {
      sums.x += __shfl_xor_sync(0xffffffffu, sums.x, s);
      sums.y += __shfl_xor_sync(0xffffffffu, sums.y, s);
    }
    if ((threadIdx.x & 31) == 0) red[parity][threadIdx.x >> 5] = sums;
    __syncthreads();
    if (threadIdx.x == 0) {
      sums = red[parity][0];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) sums = add2(sums, red[parity][i]);
      if (answers == kStealLost) sums = both(nanf(""));  // a piece may be lost: both losses say so
      if (args.cluster) block_losses = sums;
      else args.partial[piece] = sums;
    }
    parity ^= 1;
    if (next_piece < 0) break;
    round = 0;
    sums = both(0.0f);
    piece = next_piece;
    t = piece * piece_rows + group - groups;
  }
  if (!args.cluster) return;
  cluster_sync();
  if (cluster_rank() == 0 && threadIdx.x < 2) {
    double sum = 0.0;
    for (int k = 0; k < args.cluster; ++k) sum += remote_f32(threadIdx.x ? &block_losses.y : &block_losses.x, k);
    a.losses[threadIdx.x] = n > 0 ? static_cast<float>(sum * (threadIdx.x ? 1 : E) / static_cast<double>(n)) : 0.0f;
  }
  cluster_sync();  // no block leaves while another reads its sums
}

// The losses from the pieces' sums: in fp32 over each thread's pieces and the
// lanes (fp64 additions are slow on this GPU), in fp64 over the warps.
constexpr int kFinishThreads = 1024;
__global__ void __launch_bounds__(kFinishThreads) finish_kernel(const float2* __restrict__ partial, int pieces,
                                                                const int32_t* __restrict__ kept, int64_t T, int E,
                                                                float* __restrict__ losses) {
  __shared__ float2 red[kFinishThreads / 32];
  wait_for_previous();
  float2 sums = both(0.0f);
  for (int b = threadIdx.x; b < pieces; b += kFinishThreads) sums = add2(sums, partial[b]);
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    sums.x += __shfl_xor_sync(0xffffffffu, sums.x, s);
    sums.y += __shfl_xor_sync(0xffffffffu, sums.y, s);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sums;
  __syncthreads();
  if (threadIdx.x >= 2) return;
  int64_t n = T;
  if (kept) {
    n = 0;
    for (int i = 0; i < kCountBlocks; ++i) n += kept[i];
  }
  double sum = 0.0;
  for (int i = 0; i < kFinishThreads / 32; ++i) sum += threadIdx.x ? red[i].y : red[i].x;
  losses[threadIdx.x] = n > 0 ? static_cast<float>(sum * (threadIdx.x ? 1 : E) / static_cast<double>(n)) : 0.0f;
}

// After the counting kernel the losses may start early (they wait for its
// result); without it they follow the caller's work as any launch does.
template <int kValues, bool kVec, bool kFull, int kTpr>
cudaError_t launch_one(const Args& args, int grid, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr auto kernel = loss_kernel<kValues, kVec, kFull, kTpr>;
  constexpr size_t operand = kStages * (kValues / (kVec ? 4 : 1)) * static_cast<size_t>(kPitch<kVec>);
  const cudaError_t err = allow(reinterpret_cast<const void*>(kernel), done, 2 * operand, true);
  if (err != cudaSuccess) return err;
  const size_t smem = (args.a.d_in ? 2 : 1) * operand;
  if (args.cluster) return launch_cluster(kernel, args.cluster, kThreads, smem, stream, args);
  if (args.kept) return launch_dependent(kernel, grid, kThreads, smem, stream, args);
  kernel<<<grid, kThreads, smem, stream>>>(args);
  return cudaGetLastError();
}

// Only the combinations that the choice of lanes leads to: vectors with lanes
// of fewer than 8 values are a row of 4 in one lane; a full row of less than a
// warp has at most 12 values a lane.
template <bool kVec, bool kFull, int kTpr>
cudaError_t launch_losses(const Args& args, int values, int grid, cudaStream_t stream) {
  constexpr bool kFullFew = kFull && kTpr == 0;
  if constexpr (!kVec || kFullFew) {
    if (values <= 4) return launch_one<4, kVec, kFull, kTpr>(args, grid, stream);
  }
  if (values <= 8) return launch_one<8, kVec, kFull, kTpr>(args, grid, stream);
  if (kFullFew || values <= 12) return launch_one<12, kVec, kFull, kTpr>(args, grid, stream);
  if constexpr (!kFullFew) {
    if (values <= 16) return launch_one<16, kVec, kFull, kTpr>(args, grid, stream);
    return launch_one<32, kVec, kFull, kTpr>(args, grid, stream);
  }
  return cudaErrorInvalidValue;
}

// A row fills all of its lanes' values where E is so many: nothing to check;
// and a row of a whole warp then has its sizes known when compiling (65,536 x
// 384: 60.5 us without, 58.3 with).
cudaError_t launch_losses(const Args& args, bool vec, int values, int grid, cudaStream_t stream) {
  if (!vec) return launch_losses<false, false, 0>(args, values, grid, stream);
  const bool full = args.a.E == args.tpr * values && (values <= 16 || values == 32);
  if (!full) return launch_losses<true, false, 0>(args, values, grid, stream);
  return args.tpr == 32 ? launch_losses<true, true, 32>(args, values, grid, stream)
                        : launch_losses<true, true, 0>(args, values, grid, stream);
}

constexpr size_t kPartialBytes = kRouterLossMaxPieces * sizeof(float2);

}  // namespace

size_t router_loss_workspace_bytes() { return align_up(kPartialBytes + kCountBlocks * sizeof(int32_t)); }

cudaError_t launch_router_loss(const RouterLoss& a, int num_sms, cudaStream_t stream) {
  auto* kept = reinterpret_cast<int32_t*>(static_cast<char*>(a.workspace) + kPartialBytes);
  Args args{a, nullptr, static_cast<float2*>(a.workspace), 1, 0, 1, false};
  const uintptr_t low = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.d_in) |
                        reinterpret_cast<uintptr_t>(a.d_logits);
  const bool vec = a.E % 4 == 0 && low % 16 == 0;
  // few lanes with up to 12 values each (16 single ones): a row's reductions
  // cost as much as a dozen values of every lane that takes part (60,000 x 64
  // with 12 and 16 values a lane: 13.3 and 15.5 us; 65,536 x 384 with 12 and 24:
  // 56.2 and 59.8 us)
  const int units = vec ? a.E / 4 : a.E, per = vec ? 3 : 16;
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
    args.rounds = static_cast<int>((want + args.cluster - 1) / args.cluster);
    return launch_losses(args, vec, values, 0, stream);
  }
  const int64_t resident = num_sms * blocks_per_sm(values);
  int64_t rounds = (want + resident - 1) / resident;
  if (rounds >= 2 * kStealRounds) {
    args.steal = true;
    rounds = (want + kRouterLossMaxPieces - 1) / kRouterLossMaxPieces;
    if (rounds < kStealRounds) rounds = kStealRounds;
  }
  args.rounds = static_cast<int>(rounds);
  const int grid = static_cast<int>((want + rounds - 1) / rounds);
  if (a.mask) {
    args.kept = kept;
    count_kernel<<<kCountBlocks, kThreads, 0, stream>>>(a.mask, a.T, kept);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
  }
  err = launch_losses(args, vec, values, grid, stream);
  if (err != cudaSuccess) return err;
  return launch_dependent(finish_kernel, 1, kFinishThreads, 0, stream, args.partial, grid, args.kept, a.T, a.E, a.losses);
}

}  // namespace moe
