// Products of 64 inner indices of a strip of 4-bit weights (int4.cuh) with up
// to 16 rows of bf16 values, on the tensor cores.
//
// A code q becomes the bf16 value 4 + q / 4 by one AND-OR of its bits under
// the exponent of four.  (q - 8) / 4 = that - 6, so the sums of a group of
// inputs start at -6 times the sum of its inputs, which the tensor cores form
// with a constant operand for all weight rows at once; then the group's sum
// times 4 x scale, in fp32, goes to the strip's.  Codes are so multiplied
// exactly, and what cancels is at most 7 times the largest weight's share.  (Any
// power of two would do: with four, neither 4 x the largest scale that a
// quantiser can make of bf16 weights, 2^125.2, nor the sums of inputs below
// 2^118 leave the range of fp32.  An infinite input makes the sums NaN.)
#pragma once

#include "few.cuh"
#include "int4.cuh"

namespace moe {

// Bytes from a record to the scales of its first or second 64 inputs.
__device__ __forceinline__ int int4_scale_offset(int group, int second) {
  return kInt4CodeBytes + (group == 128 ? 0 : second * (64 / group) * kInt4Rows * 2);
}

__device__ __forceinline__ uint32_t int4_pair(uint32_t w, int p) {  // of input 2p and 2p + 1
  const uint32_t v = p == 0 ? w << 3 : w >> (4 * p - 3);
  return (v & 0x00780078u) | 0x40804080u;
}

// acc[tile][n][..] += tile's 16 rows x 8 columns n.  w: the codes of the 64
// inputs; groups: scales that they have, 1 or 2; rows[n]: the values of this
// lane's column, 128 bytes; low: bytes to their low parts, or 0; chunks: how
// many of the row's eight 16-byte chunks there are (the others count as zeros).
template <bool kTwo, bool kLow, int kGroups>
__device__ __forceinline__ void int4_block_of(float (&acc)[4][2][4], const uint8_t* w, const uint8_t* scales,
                                              const uint8_t* const (&rows)[2], int low, int lane, int chunks, int any_groups = 0) {
  const int groups = kGroups ? kGroups : any_groups;
  constexpr int kN = kTwo ? 2 : 1;
  constexpr uint32_t kMinus = 0xc0c0c0c0u;  // -6
  const int g = lane >> 2, t = lane & 3;
  uint4 b[2][kN];
  float start[2][kN][4];  // of inputs 0 .. 31 and 32 .. 63
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      b[c][n] = 4 * c + t < chunks ? *reinterpret_cast<const uint4*>(rows[n] + c * 64 + t * 16) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) start[c][n][i] = 0.0f;
      mma_bf16(start[c][n], kMinus, kMinus, kMinus, kMinus, b[c][n].x, b[c][n].y);
      mma_bf16(start[c][n], kMinus, kMinus, kMinus, kMinus, b[c][n].z, b[c][n].w);
      if (kLow) {
        const uint4 l = *reinterpret_cast<const uint4*>(rows[n] + low + c * 64 + t * 16);
        mma_bf16(start[c][n], kMinus, kMinus, kMinus, kMinus, l.x, l.y);
        mma_bf16(start[c][n], kMinus, kMinus, kMinus, kMinus, l.z, l.w);
      }
    }
  if (groups == 1) {  // one group: both halves' start
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) start[0][n][i] += start[1][n][i];
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const uint4 code = *reinterpret_cast<const uint4*>(w + (m * 32 + lane) * 16);
    const auto* s = reinterpret_cast<const __nv_bfloat16*>(scales) + 16 * m + g;
    float sum[kN][4];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t top = c ? code.y : code.x, bottom = c ? code.w : code.z;
      uint32_t v[4][2];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        v[p][0] = int4_pair(top, p);
        v[p][1] = int4_pair(bottom, p);
      }
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        if (c == 0 || groups == 2)
          mma_bf16_from(sum[n], start[c][n], v[0][0], v[0][1], v[1][0], v[1][1], b[c][n].x, b[c][n].y);
        else
          mma_bf16(sum[n], v[0][0], v[0][1], v[1][0], v[1][1], b[c][n].x, b[c][n].y);
        mma_bf16(sum[n], v[2][0], v[2][1], v[3][0], v[3][1], b[c][n].z, b[c][n].w);
        if (kLow) {
          const uint4 l = *reinterpret_cast<const uint4*>(rows[n] + low + c * 64 + t * 16);
          mma_bf16(sum[n], v[0][0], v[0][1], v[1][0], v[1][1], l.x, l.y);
          mma_bf16(sum[n], v[2][0], v[2][1], v[3][0], v[3][1], l.z, l.w);
        }
      }
      if (c == 1 || groups == 2) {
        const int at = groups == 2 ? c * kInt4Rows : 0;
        const float s0 = 4.0f * __bfloat162float(s[at]), s1 = 4.0f * __bfloat162float(s[at + 8]);
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] = fmaf(i < 2 ? s0 : s1, sum[n][i], acc[m][n][i]);
      }
    }
  }
}

// The same by how many scales and parts there are, which no block changes: the
// forms have no tests inside, which took 48 tokens of the 7B-A1B layer from 152
// to 144 us (moe_linear_int4's kernel has fewer registers and is better off
// with one form, 162 us where forms give 170).
template <bool kTwo>
__device__ __forceinline__ void int4_block(float (&acc)[4][2][4], const uint8_t* w, const uint8_t* scales, int groups,
                                           const uint8_t* const (&rows)[2], int low, int lane, int chunks = 8) {
  if (low) {
    if (groups == 2)
      int4_block_of<kTwo, true, 2>(acc, w, scales, rows, low, lane, chunks);
    else
      int4_block_of<kTwo, true, 1>(acc, w, scales, rows, low, lane, chunks);
  } else {
    if (groups == 2)
      int4_block_of<kTwo, false, 2>(acc, w, scales, rows, low, lane, chunks);
    else
      int4_block_of<kTwo, false, 1>(acc, w, scales, rows, low, lane, chunks);
  }
}

}  // namespace moe
