// Routing of the layer for a few tokens: top-k of each token and the list of
// units (few.cuh), in one launch.  With the router's weights given, a cluster
// of blocks computes the logits first; the first of its blocks then routes.
//
// Selection, ties and gates are moe_route_topk's.  The sets of tokens are
// 64-bit masks in shared memory, one per expert: a token takes an expert once
// at most, so a pair's place among its expert's rows is the number of lower
// bits, and no pass over pairs has an order to keep.
#include "few.cuh"
#include "internal.h"
#include "launch.cuh"
#include "route_select.cuh"

namespace moe {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kRouterBlocks = 16;  // of the cluster; a block has E_pad / 16 experts, 8 to 32
constexpr int kRouterTokens = 32;  // at a time
constexpr int kPartialPitch = kRouterTokens + 1;
constexpr size_t kRouterSmem = sizeof(float) * kWarps * 32 * kPartialPitch;

// Logits of the block's experts: [T, E_pad / 16] of x @ w_router, each warp
// a share of the 64-value K blocks.  A K block's 64 products are added by the
// tensor cores, which may cut off, the d / 1024 K blocks of a warp and the 16
// warps in fp32 registers, rounded to nearest: at most 2^-23 of the sum of
// |x| |w| for each of the 80 + d / 1024 additions that a product goes through.
__device__ __forceinline__ void router_logits(const FewRoute& p, float* partial) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int experts = p.E_pad / kRouterBlocks, e0 = static_cast<int>(cluster_rank()) * experts;
  const int nkb = p.d / 64;
  const auto* w = static_cast<const uint4*>(p.router);  // [kb][E_pad][8 chunks of 8 values]
  const auto* x = static_cast<const uint4*>(p.x);       // [T][d / 8]
  for (int t0 = 0; t0 < p.T; t0 += kRouterTokens) {
    float acc[2][4][4] = {};
    for (int kb = warp; kb < nkb; kb += kWarps) {
      uint4 a[4][2], b[4][2];
#pragma unroll
      for (int r = 0; r < 4; ++r)  // groups of 8 experts
#pragma unroll
        for (int c = 0; c < 2; ++c)
          a[r][c] = 8 * r < experts
                        ? __ldg(w + (static_cast<int64_t>(kb) * p.E_pad + e0 + 8 * r + g) * 8 + 4 * c + t)
                        : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int n = 0; n < 4; ++n)  // groups of 8 tokens
#pragma unroll
        for (int c = 0; c < 2; ++c)
          b[n][c] = t0 + 8 * n + g < p.T
                        ? __ldg(x + static_cast<int64_t>(t0 + 8 * n + g) * (p.d / 8) + kb * 8 + 4 * c + t)
                        : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          if (16 * m >= experts || t0 + 8 * n >= p.T) continue;
          float s[4] = {};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            mma_bf16(s, a[2 * m][c].x, a[2 * m + 1][c].x, a[2 * m][c].y, a[2 * m + 1][c].y, b[n][c].x, b[n][c].y);
            mma_bf16(s, a[2 * m][c].z, a[2 * m + 1][c].z, a[2 * m][c].w, a[2 * m + 1][c].w, b[n][c].z, b[n][c].w);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] += s[i];
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          partial[(warp * 32 + 16 * m + 8 * (i >> 1) + g) * kPartialPitch + 8 * n + 2 * t + (i & 1)] = acc[m][n][i];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * kRouterTokens; i += kThreads) {
      const int e = i & 31, tok = i >> 5;
      if (e < experts && e0 + e < p.E && t0 + tok < p.T) {
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) s += partial[(v * 32 + e) * kPartialPitch + tok];
        p.logits_out[static_cast<int64_t>(t0 + tok) * p.E + e0 + e] = s;
      }
    }
    __syncthreads();
  }
}

template <int NV, bool kFused>
__global__ void __launch_bounds__(kThreads, 1) few_route_kernel(const FewRoute p) {
  extern __shared__ float partial[];
  __shared__ uint64_t tokens_of[MOE_MAX_EXPERTS];
  __shared__ int32_t row_of[MOE_MAX_EXPERTS];
  __shared__ int32_t scan[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  let_next_start();
  if (kFused) {
    router_logits(p, partial);
    cluster_sync();  // the blocks' logits, in global memory
    if (cluster_rank() != 0) return;
  }
  const float* logits = kFused ? p.logits_out : p.logits;

  for (int e = tid; e < p.E; e += kThreads) tokens_of[e] = 0;
  for (int i = tid; i < p.n_counters; i += kThreads) p.counters[i] = 0;
  if (tid == 0) {
    p.header->status = 0;
    p.header->ticket = 0;
  }
  __syncthreads();
  for (int t = warp; t < p.T; t += kWarps) {
    float v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      v[i] = e < p.E ? logits[static_cast<int64_t>(t) * p.E + e] : 0.0f;
    }
    const uint64_t mine = topk_rounds<NV>(v, p.E, p.k, lane);
    const float mx = key_logit(__shfl_sync(0xffffffffu, mine, 0));
    const float z = lane < p.k ? expf(key_logit(mine) - mx) : 0.0f;
    float denom = 0.0f;
    if (p.renormalize) {
      denom = z;
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (lane + 32 * i < p.E) denom += expf(v[i] - mx);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) denom += __shfl_xor_sync(0xffffffffu, denom, s);
    denom = __shfl_sync(0xffffffffu, denom, 0);  // one rounding for every slot
    if (lane < p.k) {
      const int e = key_expert(mine);
      p.topk_idx[t * p.k + lane] = e;
      p.topk_w[t * p.k + lane] = z / denom;
      atomicOr(reinterpret_cast<unsigned long long*>(&tokens_of[e]), 1ull << t);
    }
  }
  __syncthreads();

  // units and rows before each expert: two experts a thread, both counts in
  // one word (rows below 2^16: 64 tokens of 32 experts; units are fewer)
  constexpr int kPer = MOE_MAX_EXPERTS / kThreads;
  int own[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    const int n = e < p.E ? __popcll(tokens_of[e]) : 0;
    own[i] = n + (((n + kFewChunk - 1) / kFewChunk) << 16);
    sum += own[i];
  }
  int before = sum;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, before, s);
    if (lane >= s) before += o;
  }
  if (lane == 31) scan[warp] = before;
  __syncthreads();
  before -= sum;
  for (int w = 0; w < warp; ++w) before += scan[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e < p.E) {
      uint64_t rest = tokens_of[e];
      int row = before & 0xffff, u = before >> 16;
      const int chunks = own[i] >> 16;
      row_of[e] = row;
      for (int c = 0; c < chunks; ++c) {  // kFewChunk tokens at a time
        uint64_t part = 0;
        int n = 0;
        for (; n < kFewChunk && rest; ++n) {
          part |= rest & (~rest + 1);
          rest &= rest - 1;
        }
        p.units[u++] = FewUnit{static_cast<int16_t>(e), static_cast<int8_t>(c), static_cast<int8_t>(chunks), row, part};
        row += n;
      }
    }
    before += own[i];
  }
  if (tid == kThreads - 1) p.header->n_units = before >> 16;
  __syncthreads();
  for (int i = tid; i < p.T * p.k; i += kThreads) {
    const int e = p.topk_idx[i];  // of this block's own writing
    p.pair_row[i] = row_of[e] + few_rank(tokens_of[e], i / p.k);
  }
}

template <int NV>
cudaError_t launch(const FewRoute& p, cudaStream_t stream) {
  if (!p.router) {
    few_route_kernel<NV, false><<<1, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
  }
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t err = allow(reinterpret_cast<const void*>(few_route_kernel<NV, true>), allowed, kRouterSmem, true);
  if (err != cudaSuccess) return err;
  return launch_cluster(few_route_kernel<NV, true>, kRouterBlocks, kThreads, kRouterSmem, stream, p);
}

}  // namespace

cudaError_t launch_few_route(const FewRoute& p, cudaStream_t stream) {
  const int nv = (p.E + 31) / 32;
  return nv <= 2 ? launch<2>(p, stream) : nv <= 4 ? launch<4>(p, stream) : nv <= 8 ? launch<8>(p, stream)
         : nv <= 12 ? launch<12>(p, stream) : nv <= 16 ? launch<16>(p, stream) : launch<32>(p, stream);
}

}  // namespace moe
