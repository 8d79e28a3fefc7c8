// Selection of a token's k largest logits by one warp: the keys, their order
// and the exact search that the routing kernels share.
#pragma once

#include <cstdint>

namespace moe {

// (logit, expert) as one 64-bit key whose unsigned order is the selection
// order: larger logit first, then the smaller expert index.  The high word
// is the float's bits made monotone (negative values inverted, sign bit set
// on the others) after folding -0.0 onto +0.0 (x + 0.0f: -0.0 + 0.0 is +0.0
// under round to nearest, and every other finite x is unchanged); the low
// word decreases with the expert index.  Key 0 is below every finite
// logit's key.
__device__ __forceinline__ uint32_t route_hi(float x) {
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));
  const uint32_t neg = static_cast<uint32_t>(static_cast<int32_t>(u) >> 31);  // all ones when negative
  return u ^ (neg | 0x80000000u);
}

__device__ __forceinline__ uint64_t route_key_hi(uint32_t hi, int e) {
  return (static_cast<uint64_t>(hi) << 32) | static_cast<uint32_t>(0xFFFFFFFFu - static_cast<uint32_t>(e));
}

__device__ __forceinline__ uint64_t route_key(float x, int e) { return route_key_hi(route_hi(x), e); }

__device__ __forceinline__ float key_logit(uint64_t key) {
  uint32_t u = static_cast<uint32_t>(key >> 32);
  u = (u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u;
  return __uint_as_float(u);
}

__device__ __forceinline__ int key_expert(uint64_t key) {
  return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key));
}

__device__ __forceinline__ uint64_t warp_max_u64(uint64_t b) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const uint64_t o = __shfl_xor_sync(0xffffffffu, b, s);
    b = o > b ? o : b;
  }
  return b;
}

// Bitonic sort of one key per lane over each aligned group of W lanes.
// Lanes 0 .. W-1 end in descending order (the other groups alternate in
// direction, as the network leaves them before a wider merge).
template <int W, typename Key>
__device__ __forceinline__ Key warp_sort_desc(Key v, int lane) {
#pragma unroll
  for (int size = 2; size <= W; size <<= 1) {
#pragma unroll
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      const Key o = __shfl_xor_sync(0xffffffffu, v, stride);
      const bool keep_max = ((lane & stride) == 0) == ((lane & size) == 0);
      v = keep_max ? (o > v ? o : v) : (o < v ? o : v);
    }
  }
  return v;
}

// Exact top-k of one token's keys by k rounds of warp arg-max: round j takes
// the warp maximum of the lanes' best keys, and only the lane that held it
// marks that key taken and rescans its own values.  Keys are rebuilt from
// the logits on each scan (a taken bit per value instead of a held key), so
// this rarely taken path costs no registers across the common one.  Lane
// j < k gets the j-th key.
template <int NV>
__device__ __forceinline__ uint64_t lane_best_key(const float (&v)[NV], int E, int lane, uint32_t taken) {
  uint64_t b = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    if (e < E && !((taken >> i) & 1u)) {
      const uint64_t key = route_key(v[i], e);
      b = key > b ? key : b;
    }
  }
  return b;
}

template <int NV>
__device__ __forceinline__ uint64_t topk_rounds(const float (&v)[NV], int E, int k, int lane) {
  uint32_t taken = 0;
  uint64_t lbest = lane_best_key<NV>(v, E, lane, taken);
  uint64_t mine = 0;
  for (int j = 0; j < k; ++j) {
    const uint64_t b = warp_max_u64(lbest);
    if (lane == j) mine = b;
    if (lbest == b) {  // keys are unique: exactly one lane held it
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        if (e < E && route_key(v[i], e) == b) taken |= 1u << i;
      }
      lbest = lane_best_key<NV>(v, E, lane, taken);
    }
  }
  return mine;
}

}  // namespace moe
