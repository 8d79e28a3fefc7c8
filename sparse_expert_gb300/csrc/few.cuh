// The layer for a few tokens (T <= 64): what its kernels share.
//
// A unit is one expert with up to kFewChunk of the tokens routed to it.  The
// route kernel turns the top-k selection into the list of units; everything
// after it goes by units, so an expert that no token chose costs nothing.
// The rows of a unit (one for each of its tokens, in token order) are
// consecutive in the buffers h and y.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace moe {

constexpr int kFewMaxTokens = 64;  // a set of tokens is a 64-bit mask
constexpr int kFewStrip = 32;      // fewest output features of a piece of the down projection
constexpr int kFewChunk = 16;      // tokens of a unit: two 8-column tiles of the matrix instructions

struct FewUnit {
  int16_t expert;
  int8_t chunk, chunks;  // this one of the expert's units, and how many they are (consecutive in the list)
  int32_t row;           // of the unit's first token
  uint64_t tokens;       // bit t: token t
};
static_assert(sizeof(FewUnit) == 16, "read as one vector");

// Lies over the workspace's header.
struct FewHeader {
  int32_t status;
  int32_t n_units;
  int32_t ticket;  // next piece of work of the expert kernel
  int32_t unused[61];
};
static_assert(sizeof(FewHeader) == sizeof(WsHeader), "the status word and the header's size are shared");

__device__ __forceinline__ int few_rank(uint64_t tokens, int t) {
  return __popcll(tokens & ((uint64_t(1) << t) - 1));
}

// D += A B on the tensor cores: A 16 x 16 (rows g and g + 8 of lane 4g + t),
// B 16 x 8 (column g), bf16, D fp32 (columns 2t and 2t + 1 of both rows).
// The order of the 16 inner indices is free as long as A and B agree.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same into other registers than the sums come from.
__device__ __forceinline__ void mma_bf16_from(float (&d)[4], const float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// mbar_wait_warp for waits that are often over already: the clock is read only
// where the first look fails.  kCalled: what follows that look is a call.  The
// expert kernel has a dozen of them and stalls for instructions otherwise (4 bits, 48
// tokens of the 7B-A1B layer: 140 us, 146 with all of them inlined);
// moe_linear_int4's has fewer and loses by it (13 x 6144 x 128001: 162 us, 169
// with calls).
template <int = 0>
__device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  return mbar_wait_warp_at(bar, parity, abort, limit_ns);
}
template <bool kCalled>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  if (__all_sync(0xffffffffu, mbar_try_wait(smem_addr(bar), parity))) return true;
  if constexpr (kCalled) return wait_longer(smem_addr(bar), parity, abort, limit_ns);
  return mbar_wait_warp(bar, parity, abort, limit_ns);
}

// The barrier that tells of a stage's arrival belongs to the slot and to the
// group that takes the stage: its phases are fills that this group takes, each
// of which it waits for.  (With one barrier for both groups, a ring of an odd
// number of slots gives the groups a slot's fills in turn, and a group would
// tell its next fill from its last by a parity that the other group's fill,
// not yet there, leaves unchanged.)  So the parity of a fill is that of the times
// round where the groups have slots of their own, and of half of them where
// they have them in turn.
template <int kGroups>
__device__ __forceinline__ uint32_t fill_phase(uint32_t wrap, int slots) {
  return kGroups == 1 ? wrap & 1 : (slots & 1 ? wrap >> 1 : wrap) & 1;
}

// The last thing that a fetching warp does, whether or not it fetched
// everything: waits until what it has in flight has landed (`issued` stages so
// far, into a ring of `slots`; full [kGroups][pitch]).  Its own work may be
// over while another warp gives up, and shared memory that a copy is still
// going to write must not pass to another block.
template <int kGroups, bool kCalled>
__device__ __forceinline__ void wait_for_copies(uint64_t* full, int pitch, int issued, int slots) {
  int never = 0;
  for (int n = issued < slots ? 0 : issued - slots; n < issued; ++n)
    wait_warp<kCalled>(&full[n % kGroups * pitch + n % slots], fill_phase<kGroups>(n / slots, slots), &never,
                       kWaitLimitNs);
}

}  // namespace moe
