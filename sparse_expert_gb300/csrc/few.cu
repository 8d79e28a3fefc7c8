// The experts of the layer for a few tokens: gate/up, SwiGLU, down and the
// gated sum in one persistent launch that streams the weights of the experts
// that were hit through shared memory, once.
//
// Mathematics.  For a unit (an expert and up to 16 of its tokens)
//   h = silu(x Wg) * (x Wu),  y = h Wd,  out[t] = sum_j w[t, j] y[t, j].
// Weight rows (output features) are the 16 rows of an m16n8k16 matrix
// instruction, tokens its 8 columns: with so few tokens the tensor cores have
// a fraction of their work to do, and reading the weights is the time.  h is
// kept as two bf16 (the value and what its rounding left), so that nothing but
// out is rounded to 8 bits.
//
// Work comes in pieces: kRows weight rows of a unit over the whole inner
// length (a strip), first those of the gate/up projections of all units, then
// those of down.  Blocks take pieces from a counter, in that order.  A piece of
// down waits until its unit's h is complete; whatever it waits for was taken
// earlier by a block that runs, so the wait ends whether or not all blocks are
// on the GPU at once.
//
// Behind them come pieces of the gated sum, which wait for their columns of y.
//
// Inside a block, one warp fetches weights (bulk copies into a ring of stages
// of 512 inner indices), another the tokens' rows for the same stages into a
// ring of their own, and the others multiply: each takes one 64-index block of
// a stage, for all rows and tokens, and at the end of the strip their sums are
// added in a fixed order.  A last warp tells other blocks of finished strips,
// which takes about a microsecond of waiting for memory that the multiplying
// warps so do not spend.  The weight warp does not wait for h: the next
// projection's weights are in flight while the last rows of h are being
// finished.  The inner indices are split over the warps rather than the rows,
// because every warp then reads its own part of the tokens' rows once, for all
// rows of the strip.
#include "few.cuh"
#include "int4.cuh"
#include "int4_mma.cuh"
#include "internal.h"
#include "launch.cuh"

namespace moe {
namespace {

constexpr int kStageKb = 8;                      // 64-index blocks of a stage, one for each warp of a group
constexpr int kMaxStages = 8;
constexpr int kItems = 4;                        // pieces between the weight warp and the others
constexpr int kSumCols = 64, kSumTokens = 8;     // of a piece of the gated sum
constexpr int kUnitCache = 512;                  // units kept in shared memory
constexpr size_t kSmemMost = 227 * 1024 - 1024 - sizeof(FewUnit) * kUnitCache;  // less the static variables

// Rows of a strip, groups of eight multiplying warps (a group takes every
// kGroups-th stage), and the padding of a token's row, with which the eight lanes that a 16-byte
// shared load serves at once meet different banks: two rows of 64 bytes 64
// apart, or, where a lane reads 32 bytes, 16 apart.
// Groups, one or two, as measured (us), for one token and for more of them:
// bf16 7B-A1B layer 35.2 and 37.1 (1), 215 and 229 (64), 1T layer 391 and 412
// (4); FP8 7B-A1B layer 34.7 and 34.1 (1), 1T layer 1,727 and 1,564 (32); 4 bits
// 1T layer 77.8 and 81.0 (1), 7B-A1B layer 146 and 199 (48; two groups leave 96
// registers a thread, and that kernel spills).
template <int kKind>
struct Format;
template <>
struct Format<MOE_WEIGHTS_BF16> {
  static constexpr int kRows = 32, kGroups = 1, kPad = 64;
};
template <>
struct Format<MOE_WEIGHTS_FP8> {
  static constexpr int kRows = 64, kGroups = 2, kPad = 16;
};
template <>
struct Format<MOE_WEIGHTS_INT4> {
  static constexpr int kRows = 64, kGroups = 1, kPad = 64;
};

struct Args {
  FewExperts p;
  const uint8_t *gate_up, *down;                // codes or values
  const uint8_t *gate_up_scales, *down_scales;  // FP8
  int64_t low_offset;                           // bytes from the high parts of h to the low parts
  int down_bn;                                  // rows of a packed bf16 down tile
  int cap;                                      // token rows of a stage: min(T, 16)
  int stages, stage_bytes, scale_offset;        // weights
  int row_stages, row_stage_bytes, row_offset;  // tokens' rows
  int reduce_offset;
};

__device__ __forceinline__ int32_t load_acquire(const int32_t* p) {
  int32_t v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void add_release(int32_t* p, int32_t v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Between this thread's ordinary accesses of global memory and bulk copies.
__device__ __forceinline__ void fence_proxy_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

__device__ __forceinline__ float low_f32(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_f32(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
// Two values as bf16 and what that leaves of them, also as bf16.
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& high, uint32_t& low) {
  high = pack_bf16x2(a, b);
  low = pack_bf16x2(a - low_f32(high), b - high_f32(high));
}

// A position in a ring.
struct Slot {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// Or-reduction over the multiplying warps, all of which meet here.
template <int kThreads>
__device__ __forceinline__ bool any_of(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(v ? 1u : 0u), "n"(kThreads)
      : "memory");
  return r != 0;
}

struct Piece {
  int unit, strip;
  bool down;
};

// The pieces of an expert are strip by strip, its units side by side: blocks
// that read the same weights for different tokens do so at the same time, and
// all but one of them from the L2.
__device__ __forceinline__ Piece piece_of(int i, int n_units, int strips1, int strips2, const FewUnit* units) {
  Piece q;
  q.down = i >= n_units * strips1;
  if (q.down) i -= n_units * strips1;
  const int strips = q.down ? strips2 : strips1;
  const int u = i / strips;
  const int chunks = units[u].chunks, first = u - units[u].chunk;
  const int r = i - first * strips;
  q.strip = chunks == 1 ? r : r / chunks;
  q.unit = chunks == 1 ? u : first + r % chunks;
  return q;
}

// One 64-index block of a stage: acc += rows x tokens.  `w` is the block's
// weights, `rows` the tokens' values of the same block, `low` what is to be
// added to `rows` for the low parts, or 0 where there are none.
template <int kKind>
struct Multiply;

template <>
struct Multiply<MOE_WEIGHTS_BF16> {
  // Lane 4g + t has inner indices 8t .. 8t+7 and 32 + 8t .. of its rows and
  // tokens.  Rows are 128 bytes apart, so the two rows that eight lanes read
  // at once share banks: two turns instead of one, of a shared memory whose
  // time is otherwise a third taken.
  template <bool kTwo>
  static __device__ __forceinline__ void block(float (&acc)[2][2][4], const uint8_t* w, const uint8_t*, int, int,
                                               const uint8_t* const (&rows)[2], int low, int lane) {
    constexpr int kHalf = Format<MOE_WEIGHTS_BF16>::kRows / 2 * 128;
    const int g = lane >> 2, t = lane & 3;
    uint4 a[2][2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          a[m][half][c] = *reinterpret_cast<const uint4*>(w + half * kHalf + (8 * m + g) * 128 + c * 64 + t * 16);
    for (int part = 0;; part = low) {
#pragma unroll
      for (int n = 0; n < (kTwo ? 2 : 1); ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 b = *reinterpret_cast<const uint4*>(rows[n] + part + c * 64 + t * 16);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            mma_bf16(acc[m][n], a[m][0][c].x, a[m][1][c].x, a[m][0][c].y, a[m][1][c].y, b.x, b.y);
            mma_bf16(acc[m][n], a[m][0][c].z, a[m][1][c].z, a[m][0][c].w, a[m][1][c].w, b.z, b.w);
          }
        }
      if (part == low) break;
    }
  }
};

// E4M3 codes become bf16 by moving their bits: the code's sign, four exponent
// bits and three mantissa bits at bf16's places are the code's value times
// 2^-120, exactly, subnormal codes included.  The inputs carry 2^60 against
// that, and the sums the other 2^60 at the end: inputs times scale may be up to
// 2^67 in size, and products go down to 2^-66 before they lose bits.  (Beyond,
// the value is infinite and its remainder NaN: to test for that here takes the
// batch of 32 tokens from 1,551 to 1,602-1,644 us.)  Scales belong to an inner index (and 128 output features), so they
// are multiplied into the inputs, once for all rows of the strip; the fp32
// products enter as two bf16 each, which keeps 16 bits of them.
constexpr float kFp8Lift = 1.152921504606846976e18f;  // 2^60

template <>
struct Multiply<MOE_WEIGHTS_FP8> {
  // Lane 4g + t has inner indices 16t .. 16t+15: 16 codes of a row.  Word i
  // of them is the operand of one instruction: bytes 0 and 2, and 1 and 3.
  template <bool kTwo>
  static __device__ __forceinline__ void block(float (&acc)[4][2][4], const uint8_t* w, const uint8_t* scales, int down,
                                               int, const uint8_t* const (&rows)[2], int low, int lane) {
    const int g = lane >> 2, t = lane & 3;
    // gate and up tiles alternate and have scales of their own
    for (int proj = 0; proj < (down ? 1 : 2); ++proj) {
      uint32_t bh[2][8], bl[2][8];
      const auto* s = reinterpret_cast<const float4*>(scales + proj * 272) + 4 * t;
#pragma unroll
      for (int n = 0; n < (kTwo ? 2 : 1); ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 sc = s[i];
          const uint2 hi = *reinterpret_cast<const uint2*>(rows[n] + t * 32 + i * 8);
          float v[4] = {low_f32(hi.x), high_f32(hi.x), low_f32(hi.y), high_f32(hi.y)};
          if (low) {
            const uint2 lo = *reinterpret_cast<const uint2*>(rows[n] + low + t * 32 + i * 8);
            v[0] += low_f32(lo.x);
            v[1] += high_f32(lo.x);
            v[2] += low_f32(lo.y);
            v[3] += high_f32(lo.y);
          }
          v[0] *= kFp8Lift * sc.x;
          v[1] *= kFp8Lift * sc.y;
          v[2] *= kFp8Lift * sc.z;
          v[3] *= kFp8Lift * sc.w;
          split_bf16(v[0], v[2], bh[n][2 * i], bl[n][2 * i]);
          split_bf16(v[1], v[3], bh[n][2 * i + 1], bl[n][2 * i + 1]);
        }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (!down && (m & 1) != proj) continue;
        const uint4 c0 = *reinterpret_cast<const uint4*>(w + (16 * m + g) * 64 + t * 16);
        const uint4 c1 = *reinterpret_cast<const uint4*>(w + (16 * m + 8 + g) * 64 + t * 16);
        const uint32_t top[4] = {c0.x, c0.y, c0.z, c0.w}, bottom[4] = {c1.x, c1.y, c1.z, c1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = even(top[i]), a1 = even(bottom[i]), a2 = odd(top[i]), a3 = odd(bottom[i]);
#pragma unroll
          for (int n = 0; n < (kTwo ? 2 : 1); ++n) {
            mma_bf16(acc[m][n], a0, a1, a2, a3, bh[n][2 * i], bh[n][2 * i + 1]);
            mma_bf16(acc[m][n], a0, a1, a2, a3, bl[n][2 * i], bl[n][2 * i + 1]);
          }
        }
      }
    }
  }
  static __device__ __forceinline__ uint32_t even(uint32_t c) {  // bytes 0 and 2
    return ((c << 8) & 0x80008000u) | ((c << 4) & 0x07f007f0u);
  }
  static __device__ __forceinline__ uint32_t odd(uint32_t c) {  // bytes 1 and 3
    return (c & 0x80008000u) | ((c >> 4) & 0x07f007f0u);
  }
};

template <>
struct Multiply<MOE_WEIGHTS_INT4> {
  template <bool kTwo>
  static __device__ __forceinline__ void block(float (&acc)[4][2][4], const uint8_t* w, const uint8_t* scales, int,
                                               int groups, const uint8_t* const (&rows)[2], int low, int lane) {
    int4_block<kTwo>(acc, w, scales, groups, rows, low, lane);
  }
};

template <int kKind>
__global__ void __launch_bounds__((Format<kKind>::kGroups * 8 + 3) * 32, 1) few_experts_kernel(const Args a) {
  using F = Format<kKind>;
  constexpr int kRows = F::kRows, kTiles = kRows / 16, kWarps = F::kGroups * 8, kThreads = kWarps * 32;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full_w[F::kGroups][kMaxStages], empty_w[kMaxStages];
  __shared__ uint64_t full_x[F::kGroups][kMaxStages], empty_x[kMaxStages];
  __shared__ uint64_t item_full[kItems], item_done[kItems], item_empty[kItems];
  __shared__ int32_t item[kItems];
  __shared__ __align__(16) FewUnit unit_cache[kUnitCache];
  __shared__ int abort_s, n_units_s, first_s;
  const FewExperts& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &abort_s;

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      for (int j = 0; j < F::kGroups; ++j) mbar_init(&full_w[j][i], 1);
      mbar_init(&empty_w[i], 8);
    }
    for (int i = 0; i < a.row_stages; ++i) {
      for (int j = 0; j < F::kGroups; ++j) mbar_init(&full_x[j][i], 1);
      mbar_init(&empty_x[i], 8);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_done[i], kWarps);
      mbar_init(&item_empty[i], 2 + kWarps);
    }
    abort_s = 0;
    fence_barrier_init();
  }
  wait_for_previous();
  // the units, as many as there can be, beside the number that there are and
  // the first piece: one latency for the three
  const int most = p.T * p.k;
  for (int i = threadIdx.x; i < most && i < kUnitCache; i += blockDim.x)
    reinterpret_cast<uint4*>(unit_cache)[i] = reinterpret_cast<const uint4*>(p.units)[i];
  if (threadIdx.x == 0) {
    first_s = atomicAdd(&p.header->ticket, 1);
    n_units_s = p.header->n_units;
  }
  __syncthreads();
  const FewUnit* units = most <= kUnitCache ? unit_cache : p.units;
  const int n_units = n_units_s;
  const int strips1 = 2 * p.f / kRows, strips2 = p.d / kRows;
  const int products = n_units * (strips1 + strips2);  // pieces
  const int sum_groups = (p.T + kSumTokens - 1) / kSumTokens, total = products + p.d / kSumCols * sum_groups;
  const int kb1 = p.d / 64, kb2 = p.f / 64;
  constexpr int kPitch = kStageKb * 128 + F::kPad;
  bool ok = true;

  if (warp == kWarps) {
    // ------------------------------------------------ weights
    Slot st, it;
    int issued = 0;
    for (int i = first_s;;) {
      int next = 0;
      if (lane == 0) next = atomicAdd(&p.header->ticket, 1);
      ok = wait_warp<true>(&item_empty[it.slot], it.phase ^ 1, abort, p.wait_ns);
      if (!ok) break;
      if (lane == 0) {
        item[it.slot] = i < total ? i : -1;
        mbar_arrive(&item_full[it.slot]);
      }
      it.next(kItems);
      if (i >= total) break;
      if (i >= products) {
        i = __shfl_sync(0xffffffffu, next, 0);
        continue;
      }
      const Piece q = piece_of(i, n_units, strips1, strips2, units);
      const int e = units[q.unit].expert, nkb = q.down ? kb2 : kb1;
      for (int kb0 = 0; kb0 < nkb; kb0 += kStageKb) {
        const int nk = min(kStageKb, nkb - kb0);
        ok = wait_warp<true>(&empty_w[st.slot], st.phase ^ 1, abort, p.wait_ns);
        if (!ok) break;
        uint8_t* dst = ring + st.slot * a.stage_bytes;
        uint64_t* bar = &full_w[issued % F::kGroups][st.slot];
        if (kKind == MOE_WEIGHTS_BF16) {
          // packed tiles of 128 (gate/up: 64 and 64) or down_bn rows of 64
          // values; two runs of kRows / 2 rows for each 64-index block
          constexpr int kRun = kRows / 2 * 128;
          if (lane == 0) mbar_arrive_expect_tx(bar, nk * 2 * kRun);
          __syncwarp();
          if (lane < 2 * nk) {
            const int half = lane & 1, kb = kb0 + (lane >> 1);
            const int bn = q.down ? a.down_bn : 128, tiles = (q.down ? p.d : 2 * p.f) / bn;
            const int row = q.down ? q.strip * kRows + half * (kRows / 2)
                                   : q.strip * (kRows / 2) / 64 * 128 + half * 64 + q.strip * (kRows / 2) % 64;
            const uint8_t* src = (q.down ? a.down : a.gate_up) +
                                 (((static_cast<int64_t>(e) * tiles + row / bn) * nkb + kb) * bn + row % bn) * 128;
            bulk_load(dst + lane * kRun, src, kRun, bar);
          }
        } else if (kKind == MOE_WEIGHTS_FP8) {
          // packed tiles of 128 rows of 64 codes, and the scales of the
          // blocks (gate and up, or down) of the strip's 128 features
          constexpr int kRun = kRows * 64;
          const int record = (q.down ? kFp8DownRecord : kFp8GateUpRecord) * 4;
          if (lane == 0) mbar_arrive_expect_tx(bar, nk * (kRun + record));
          __syncwarp();
          const int tiles = (q.down ? p.d : 2 * p.f) / 128, row = q.strip * kRows;
          if (lane < nk)
            bulk_load(dst + lane * kRun,
                      (q.down ? a.down : a.gate_up) +
                          (((static_cast<int64_t>(e) * tiles + row / 128) * nkb + kb0 + lane) * 128 + row % 128) * 64,
                      kRun, bar);
          if (lane == 31) {
            const int blocks = (q.down ? p.d : p.f) / 128, fb = q.down ? row / 128 : row / 256;
            bulk_load(dst + a.scale_offset,
                      (q.down ? a.down_scales : a.gate_up_scales) +
                          ((static_cast<int64_t>(e) * blocks + fb) * nkb + kb0) * record,
                      nk * record, bar);
          }
        } else {
          const int record = int4_record_bytes(p.group), bytes = nk / 2 * record;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, bytes);
            const int64_t strip = static_cast<int64_t>(e) * (q.down ? strips2 : strips1) + q.strip;
            bulk_load(dst, (q.down ? a.down : a.gate_up) + (strip * (nkb / 2) + kb0 / 2) * record, bytes, bar);
          }
        }
        ++issued;
        st.next(a.stages);
      }
      if (!ok) break;
      i = __shfl_sync(0xffffffffu, next, 0);
    }
    if (!ok) abort_s = 1;
    wait_for_copies<F::kGroups, true>(full_w[0], kMaxStages, issued, a.stages);
  } else if (warp == kWarps + 1) {
    // ------------------------------------------------ the tokens' rows
    Slot st, it;
    int issued = 0, complete = -1;
    while (ok) {
      ok = wait_warp<true>(&item_full[it.slot], it.phase, abort, p.wait_ns);
      if (!ok) break;
      const int i = *reinterpret_cast<volatile int32_t*>(&item[it.slot]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[it.slot]);
      it.next(kItems);
      if (i < 0) break;
      if (i >= products) continue;
      const Piece q = piece_of(i, n_units, strips1, strips2, units);
      const FewUnit u = units[q.unit];
      const int n = __popcll(u.tokens), nkb = q.down ? kb2 : kb1, parts = q.down ? 2 : 1;
      if (q.down && complete != q.unit) {  // every strip of its h
        const uint64_t t0 = global_timer_ns();
        while (load_acquire(p.ready + q.unit) != strips1) {
          if (*abort || global_timer_ns() - t0 > p.wait_ns) {
            ok = false;
            break;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        fence_proxy_global();
        complete = q.unit;
      }
      // lane j: row j of the unit, lane 16 + j: the low part of it
      const int j = lane & 15, part = lane >> 4;
      const uint8_t* src = nullptr;
      if (j < n && part < parts) {
        if (q.down) {
          src = static_cast<const uint8_t*>(p.h) + part * a.low_offset + static_cast<int64_t>(u.row + j) * p.f * 2;
        } else {
          uint64_t rest = u.tokens;
          for (int s = 0; s < j; ++s) rest &= rest - 1;
          const int token = __ffsll(static_cast<long long>(rest)) - 1;
          src = static_cast<const uint8_t*>(p.x) + static_cast<int64_t>(token) * p.d * 2;
        }
      }
      uint8_t* dst = ring + a.row_offset + (part * a.cap + j) * kPitch;
      for (int kb0 = 0; kb0 < nkb; kb0 += kStageKb) {
        const int bytes = min(kStageKb, nkb - kb0) * 128;
        ok = wait_warp<true>(&empty_x[st.slot], st.phase ^ 1, abort, p.wait_ns);
        if (!ok) break;
        uint64_t* bar = &full_x[issued % F::kGroups][st.slot];
        if (lane == 0) mbar_arrive_expect_tx(bar, n * parts * bytes);
        __syncwarp();
        if (src) bulk_load(dst + st.slot * a.row_stage_bytes, src + kb0 * 128, bytes, bar);
        ++issued;
        st.next(a.row_stages);
      }
    }
    if (!ok) abort_s = 1;
    wait_for_copies<F::kGroups, true>(full_x[0], kMaxStages, issued, a.row_stages);
  } else if (warp == kWarps + 2) {
    // ------------------------------------------------ news of finished strips
    Slot it;
    while (ok) {
      ok = wait_warp<true>(&item_full[it.slot], it.phase, abort, p.wait_ns);
      if (!ok) break;
      const int i = *reinterpret_cast<volatile int32_t*>(&item[it.slot]);
      if (i >= 0 && i < products) {
        ok = wait_warp<true>(&item_done[it.slot], it.phase, abort, p.wait_ns);
        if (!ok) break;
        const Piece q = piece_of(i, n_units, strips1, strips2, units);
        if (lane == 0) add_release(q.down ? p.strips + q.strip : p.ready + q.unit, 1);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[it.slot]);
      it.next(kItems);
      if (i < 0) break;
    }
    if (!ok) abort_s = 1;
  } else {
    // ------------------------------------------------ products
    const int group = warp >> 3, kb_own = warp & 7, g = lane >> 2, t = lane & 3;
    Slot st, row_st, it;
    uint32_t own_w = 0, own_x = 0;  // two groups: bit i is the phase of this group's barrier of slot i
    int turn = 0, buffer = 0;  // of the groups; of the sums
    float* const reduce = reinterpret_cast<float*>(ring + a.reduce_offset);  // [2][8 warps][kRows][8]
    for (;;) {
      // A wait that ran out in one warp ends all of them, together: they meet
      // at the next or-reduction, one for each piece of a product and one at
      // the end, and none waits for a barrier that another does not reach.
      if (ok) ok = wait_warp<true>(&item_full[it.slot], it.phase, abort, p.wait_ns);
      if (!ok) {
        abort_s = 1;
        if (F::kGroups == 2 && group == 0) asm volatile("barrier.cta.arrive %0, 64;" ::"r"(2 + kb_own) : "memory");
        any_of<kThreads>(true);
        break;
      }
      const int slot = it.slot, i = *reinterpret_cast<volatile int32_t*>(&item[slot]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[slot]);
      it.next(kItems);
      if (i < 0) {
        ok = !any_of<kThreads>(false);
        break;
      }
      if (i >= products) {
        // the gated sum of some columns of some tokens, once every unit has
        // its part of them
        const int col0 = (i - products) / sum_groups * kSumCols, t0 = (i - products) % sum_groups * kSumTokens;
        const uint64_t begin = global_timer_ns();
        for (int s = col0 / kRows; s * kRows < col0 + kSumCols; ++s)
          while (ok && load_acquire(p.strips + s) != n_units)
            if (*abort || global_timer_ns() - begin > p.wait_ns) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        for (int o = threadIdx.x; o < kSumCols * min(kSumTokens, p.T - t0); o += kThreads) {
          const int token = t0 + o / kSumCols, n = col0 + o % kSumCols;
          float s = 0.0f;
#pragma unroll 8
          for (int j = 0; j < p.k; ++j) {
            // written by the previous launch while this one's blocks are
            // already there: plain loads, not the read-only path
            const float w = p.topk_w[token * p.k + j];
            const int row = p.pair_row[token * p.k + j];
            s = fmaf(w, __ldcg(p.y + static_cast<int64_t>(row) * p.d + n), s);
          }
          static_cast<__nv_bfloat16*>(p.out)[static_cast<int64_t>(token) * p.d + n] = __float2bfloat16_rn(s);
        }
        continue;
      }
      const Piece q = piece_of(i, n_units, strips1, strips2, units);
      const FewUnit u = units[q.unit];
      const int n_tok = __popcll(u.tokens), nkb = q.down ? kb2 : kb1;
      const bool two = n_tok > 8;
      float acc[kTiles][2][4] = {};
      for (int kb0 = 0; kb0 < nkb; kb0 += kStageKb) {
        if (turn == group) {
          // (calls only in kernels of one group: FP8, 64 tokens of the 7B-A1B
          // layer, 199 us, 203 with calls)
          constexpr bool kCalled = F::kGroups == 1;
          const uint32_t phase_x = F::kGroups == 1 ? row_st.phase : own_x >> row_st.slot & 1;
          const uint32_t phase_w = F::kGroups == 1 ? st.phase : own_w >> st.slot & 1;
          ok = wait_warp<kCalled>(&full_x[group][row_st.slot], phase_x, abort, p.wait_ns);
          if (ok) ok = wait_warp<kCalled>(&full_w[group][st.slot], phase_w, abort, p.wait_ns);
          own_x ^= 1u << row_st.slot;
          own_w ^= 1u << st.slot;
          if (!ok) {
            abort_s = 1;
            break;
          }
          if (kb_own < nkb - kb0) {
            const uint8_t* base = ring + st.slot * a.stage_bytes;
            const uint8_t* w;
            const uint8_t* scales = nullptr;
            int groups = 0;
            if (kKind == MOE_WEIGHTS_BF16) {
              w = base + kb_own * kRows * 128;
            } else if (kKind == MOE_WEIGHTS_FP8) {
              w = base + kb_own * kRows * 64;
              scales = base + a.scale_offset + kb_own * (q.down ? kFp8DownRecord : kFp8GateUpRecord) * 4;
            } else {
              const uint8_t* record = base + kb_own / 2 * int4_record_bytes(p.group);
              w = record + (kb_own & 1) * (kInt4CodeBytes / 2);
              groups = p.group == 32 ? 2 : 1;
              scales = record + int4_scale_offset(p.group, kb_own & 1);
            }
            // columns without a token read the first one's row
            const uint8_t* r0 = ring + a.row_offset + row_st.slot * a.row_stage_bytes + kb_own * 128;
            const uint8_t* const rows[2] = {r0 + (g < n_tok ? g : 0) * kPitch, r0 + (8 + g < n_tok ? 8 + g : 0) * kPitch};
            const int low = q.down ? a.cap * kPitch : 0;
            if (two)
              Multiply<kKind>::template block<true>(acc, w, scales, q.down, groups, rows, low, lane);
            else
              Multiply<kKind>::template block<false>(acc, w, scales, q.down, groups, rows, low, lane);
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&empty_w[st.slot]);
            mbar_arrive(&empty_x[row_st.slot]);
          }
        }
        st.next(a.stages);
        row_st.next(a.row_stages);
        if (++turn == F::kGroups) turn = 0;
      }
      bool lost = false;
      for (int n = 0; n < (two ? 2 : 1) && !lost; ++n) {
        // Eight partial sums of every value, the second group's added to the
        // first's.  A buffer is written again after the next barrier but one
        // at the earliest, when all have read it.
        float* const sums = reduce + buffer * (8 * kRows * 8);
        buffer ^= 1;
        if (F::kGroups == 2 && group == 1) asm volatile("barrier.cta.sync %0, 64;" ::"r"(2 + kb_own) : "memory");
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int row = kKind == MOE_WEIGHTS_BF16 ? half * (kRows / 2) + 8 * m + g : 16 * m + 8 * half + g;
            float2 v = n == 0 ? make_float2(acc[m][0][2 * half], acc[m][0][2 * half + 1])
                              : make_float2(acc[m][1][2 * half], acc[m][1][2 * half + 1]);
            auto* to = reinterpret_cast<float2*>(sums + (kb_own * kRows + row) * 8 + 2 * t);
            if (F::kGroups == 2 && group == 1) {
              v.x += to->x;
              v.y += to->y;
            }
            *to = v;
          }
        if (F::kGroups == 2 && group == 0) asm volatile("barrier.cta.arrive %0, 64;" ::"r"(2 + kb_own) : "memory");
        lost = any_of<kThreads>(!ok);
        constexpr float kLift = kKind == MOE_WEIGHTS_FP8 ? kFp8Lift : 1.0f;
        const int tok = 8 * n + (threadIdx.x & 7);
        if (tok < n_tok && !lost) {
          const float* own = sums + (threadIdx.x & 7);
          if (!q.down) {
            for (int feature = threadIdx.x >> 3; feature < kRows / 2; feature += kThreads / 8) {
              const int row = kKind == MOE_WEIGHTS_FP8 ? feature / 16 * 32 + feature % 16 : feature;
              constexpr int kToUp = kKind == MOE_WEIGHTS_FP8 ? 16 : kRows / 2;
              float gate = 0.0f, up = 0.0f;
#pragma unroll
              for (int v = 0; v < 8; ++v) {
                gate += own[(v * kRows + row) * 8];
                up += own[(v * kRows + row + kToUp) * 8];
              }
              gate *= kLift;
              up *= kLift;
              const float h = gate / (1.0f + __expf(-gate)) * up;
              const int64_t at = static_cast<int64_t>(u.row + tok) * p.f + q.strip * (kRows / 2) + feature;
              // Rounded to nearest, the largest finite values would become
              // infinite: their high part is cut off instead.  An infinity has
              // no remainder (its difference from itself would be NaN).
              __nv_bfloat16 high = __float2bfloat16_rn(h);
              if (isinf(__bfloat162float(high))) high = __float2bfloat16_rz(h);
              auto* to = static_cast<__nv_bfloat16*>(p.h);
              to[at] = high;
              to[a.low_offset / 2 + at] = __float2bfloat16_rn(isinf(h) ? 0.0f : h - __bfloat162float(high));
            }
          } else {
            for (int row = threadIdx.x >> 3; row < kRows; row += kThreads / 8) {
              float y = 0.0f;
#pragma unroll
              for (int v = 0; v < 8; ++v) y += own[(v * kRows + row) * 8];
              p.y[static_cast<int64_t>(u.row + tok) * p.d + q.strip * kRows + row] = y * kLift;
            }
          }
        }
      }
      if (lost) {
        ok = false;
        break;
      }
      if (!q.down) fence_proxy_global();  // h is read by bulk copies
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_done[slot]);
    }
  }
  if (!ok && lane == 0) record_status(&p.header->status, kStatusTimeout);
}

template <int kKind>
cudaError_t launch(Args& a, int weight_bytes, int scale_bytes, int num_sms, cudaStream_t stream) {
  using F = Format<kKind>;
  constexpr int kReduce = 2 * 8 * F::kRows * 8 * 4;
  a.scale_offset = weight_bytes;
  a.stage_bytes = static_cast<int>(align_up(weight_bytes + scale_bytes, 128));
  a.row_stage_bytes = static_cast<int>(align_up(2 * a.cap * (kStageKb * 128 + F::kPad), 128));
  // rows come from the L2 and need fewer stages in flight than weights do
  a.row_stages = a.cap <= 4 ? 4 : a.cap <= 8 ? 3 : 2;
  const int rest = static_cast<int>(kSmemMost) - kReduce - a.row_stages * a.row_stage_bytes;
  a.stages = rest / a.stage_bytes < kMaxStages ? rest / a.stage_bytes : kMaxStages;
  a.row_offset = a.stages * a.stage_bytes;
  a.reduce_offset = a.row_offset + a.row_stages * a.row_stage_bytes;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t err = allow(reinterpret_cast<const void*>(few_experts_kernel<kKind>), allowed, kSmemMost, false);
  if (err != cudaSuccess) return err;
  return launch_dependent(few_experts_kernel<kKind>, dim3(num_sms), dim3((F::kGroups * 8 + 3) * 32),
                          a.reduce_offset + kReduce, stream, a);
}

}  // namespace

cudaError_t launch_few_experts(const FewExperts& p, int num_sms, cudaStream_t stream) {
  Args a{};
  a.p = p;
  a.cap = p.T < kFewChunk ? p.T : kFewChunk;
  a.low_offset = static_cast<int64_t>(p.T) * p.k * p.f * 2;
  const auto* packed = static_cast<const uint8_t*>(p.packed);
  const int64_t edf = static_cast<int64_t>(p.E) * p.d * p.f;
  switch (p.weights) {
    case MOE_WEIGHTS_BF16:
      a.gate_up = packed;
      a.down = packed + 4 * edf;
      a.down_bn = down_tile_n(p.d);
      return launch<MOE_WEIGHTS_BF16>(a, kStageKb * Format<MOE_WEIGHTS_BF16>::kRows * 128, 0, num_sms, stream);
    case MOE_WEIGHTS_FP8: {
      size_t off[4];
      fp8_packed_bytes(p.E, p.d, p.f, off);
      a.gate_up = packed + off[0];
      a.down = packed + off[1];
      a.gate_up_scales = packed + off[2];
      a.down_scales = packed + off[3];
      return launch<MOE_WEIGHTS_FP8>(a, kStageKb * Format<MOE_WEIGHTS_FP8>::kRows * 64, kStageKb * kFp8GateUpRecord * 4,
                                     num_sms, stream);
    }
    default:
      a.gate_up = packed;
      a.down = packed + align_up(int4_matrix_bytes(p.E, p.d, 2 * static_cast<int64_t>(p.f), p.group));
      return launch<MOE_WEIGHTS_INT4>(a, kStageKb / 2 * int4_record_bytes(p.group), 0, num_sms, stream);
  }
}

}  // namespace moe
