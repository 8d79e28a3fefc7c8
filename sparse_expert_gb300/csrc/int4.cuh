// The packed layout of 4-bit weights, made for the kernels that read it: a
// record (kInt4Rows output features x kInt4Unit inputs) is one contiguous
// piece of memory, and a thread reads its codes for a matrix instruction's
// operand as whole 16-byte words, without bank conflicts.
//
//   record (matrix, strip, unit), units of a strip one after the other:
//     codes   [2 K blocks of 64][4 tiles of 16 rows][32 lanes][16 bytes]
//     scales  [kInt4Unit / group][kInt4Rows] bf16
//   Lane 4g + t of a tile has rows g (8 bytes) and g + 8 (8 bytes); of each,
//   inputs 8t .. 8t+7 of the K block in the first word and 32 + 8t .. in the
//   second.  Input 2p of a word is in bits 4p .. 4p+3 and input 2p + 1 in bits
//   4p+16 .. 4p+19, so (word >> 4p) & 0x000f000f is a pair of neighbours.
//   A strip's rows: 64 output features, or for gate/up 32 gate features and
//   then the same 32 up features.  Features beyond N and inputs beyond K have
//   code 8 and scale 0.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace moe {

constexpr int kInt4Rows = 64;
constexpr int kInt4Unit = 128;
constexpr int kInt4CodeBytes = kInt4Rows * kInt4Unit / 2;

__host__ __device__ constexpr int int4_record_bytes(int group) {
  return kInt4CodeBytes + kInt4Unit / group * kInt4Rows * 2;
}

}  // namespace moe
