// Products of a few rows with 4-bit weights: y = x W, M <= 16.
//
// As in the experts of the layer for a few tokens, the output features are the
// rows of the matrix instructions and the M rows their columns, and the bytes
// of the weights are the time.  A block has a strip of 64 output features: one
// warp fetches records of codes and scales into a ring of stages of 512 inputs,
// one the rows of x for them, and eight multiply, each a 64-input block of a
// stage for the whole strip; their sums are added in a fixed order.  Two
// blocks share an SM, so that one's ends are hidden by the other.
//
// Matrices with many strips are walked by blocks that stay (strip after strip,
// the next one's weights in flight during the sums of the last).  Where strips
// are no more than the SMs, the inputs of a strip are split over a cluster's
// blocks instead, which add their sums through each other's shared memory: no
// scratch in memory, and no order that could change a result.
#include "int4.cuh"
#include "int4_mma.cuh"
#include "internal.h"
#include "launch.cuh"

namespace moe {
namespace {

constexpr int kStageKb = 8, kStageUnits = kStageKb * 64 / kInt4Unit;
constexpr int kStages = 3, kRowStages = 2;
constexpr int kPitch = kStageKb * 128 + 64;
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kReduce = kWarps * kInt4Rows * 8 * 4;  // of 8 columns
constexpr int kMostSplit = 8;

struct Args {
  LinearInt4 p;
  int strips, units, units_per_rank, split;
  int stage_bytes, row_offset, row_stage_bytes, reduce_offset, part_offset;
};

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

__global__ void __launch_bounds__((kWarps + 2) * 32, 2) linear_int4_kernel(const Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full_w[kStages], empty_w[kStages], full_x[kRowStages], empty_x[kRowStages];
  __shared__ int abort_s;
  const LinearInt4& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &abort_s;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full_w[i], 1);
      mbar_init(&empty_w[i], kWarps);
    }
    for (int i = 0; i < kRowStages; ++i) {
      mbar_init(&full_x[i], 1);
      mbar_init(&empty_x[i], kWarps);
    }
    abort_s = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const int rank = a.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int first = blockIdx.x / a.split, step = gridDim.x / a.split;
  const int unit0 = rank * a.units_per_rank, unit1 = min(a.units, unit0 + a.units_per_rank);
  const int record = int4_record_bytes(p.group);
  // sums of this block, [64][16]; with one block a strip they go to out at once
  float* const part = reinterpret_cast<float*>(smem + a.part_offset);
  bool ok = true;

  if (warp == kWarps) {
    Slot st;
    int issued = 0;
    for (int strip = first; strip < a.strips && ok; strip += step)
      for (int u = unit0; u < unit1; u += kStageUnits) {
        ok = wait_warp<false>(&empty_w[st.slot], st.phase ^ 1, abort, p.wait_ns);
        if (!ok) break;
        if (lane == 0) {
          const int bytes = min(kStageUnits, unit1 - u) * record;
          mbar_arrive_expect_tx(&full_w[st.slot], bytes);
          bulk_load(smem + st.slot * a.stage_bytes,
                    static_cast<const uint8_t*>(p.packed) + (static_cast<int64_t>(strip) * a.units + u) * record, bytes,
                    &full_w[st.slot]);
        }
        ++issued;
        st.next(kStages);
      }
    if (!ok) abort_s = 1;
    wait_for_copies<1, false>(full_w, kStages, issued, kStages);
  } else if (warp == kWarps + 1) {
    Slot st;
    int issued = 0;
    const uint8_t* src = lane < p.M ? static_cast<const uint8_t*>(p.x) + lane * p.x_stride * 2 : nullptr;
    for (int strip = first; strip < p.row_strips && ok; strip += step)
      for (int u = unit0; u < unit1; u += kStageUnits) {
        ok = wait_warp<false>(&empty_x[st.slot], st.phase ^ 1, abort, p.wait_ns);
        if (!ok) break;
        const int k0 = u * kInt4Unit, bytes = 2 * (min(p.K, min(unit1, u + kStageUnits) * kInt4Unit) - k0);
        if (lane == 0) mbar_arrive_expect_tx(&full_x[st.slot], p.M * bytes);
        __syncwarp();
        if (src)
          bulk_load(smem + a.row_offset + st.slot * a.row_stage_bytes + lane * kPitch, src + 2 * k0, bytes,
                    &full_x[st.slot]);
        ++issued;
        st.next(kRowStages);
      }
    if (!ok) abort_s = 1;
    wait_for_copies<1, false>(full_x, kRowStages, issued, kRowStages);
  } else {
    const int g = lane >> 2, t = lane & 3;
    const bool two = p.M > 8;
    float* const sums = reinterpret_cast<float*>(smem + a.reduce_offset);  // [warp][64][8]
    Slot st, row_st;
    for (int strip = first; strip < a.strips; strip += step) {
      float acc[4][2][4] = {};
      for (int u = unit0; u < unit1 && ok; u += kStageUnits) {
        ok = wait_warp<false>(&full_x[row_st.slot], row_st.phase, abort, p.wait_ns);
        if (ok) ok = wait_warp<false>(&full_w[st.slot], st.phase, abort, p.wait_ns);
        if (!ok) {
          abort_s = 1;
          break;
        }
        const int left = p.K - (u * kInt4Unit + warp * 64);  // inputs from this warp's block on
        if (left > 0 && warp / 2 < unit1 - u) {
          const uint8_t* r = smem + st.slot * a.stage_bytes + warp / 2 * record;
          const uint8_t* r0 = smem + a.row_offset + row_st.slot * a.row_stage_bytes + warp * 128;
          const uint8_t* const rows[2] = {r0 + (g < p.M ? g : 0) * kPitch, r0 + (8 + g < p.M ? 8 + g : 0) * kPitch};
          const uint8_t* codes = r + (warp & 1) * (kInt4CodeBytes / 2);
          const uint8_t* scales = r + int4_scale_offset(p.group, warp & 1);
          const int groups = p.group == 32 ? 2 : 1, chunks = left / 8;
          if (two)
            int4_block_of<true, false, 0>(acc, codes, scales, rows, 0, lane, chunks, groups);
          else
            int4_block_of<false, false, 0>(acc, codes, scales, rows, 0, lane, chunks, groups);
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&empty_w[st.slot]);
          mbar_arrive(&empty_x[row_st.slot]);
        }
        st.next(kStages);
        row_st.next(kRowStages);
      }
      for (int n = 0; n < (two ? 2 : 1); ++n) {
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float2 v = n == 0 ? make_float2(acc[m][0][2 * half], acc[m][0][2 * half + 1])
                              : make_float2(acc[m][1][2 * half], acc[m][1][2 * half + 1]);
            // a wait that ran out shows as NaN
            if (!ok) v = make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
            *reinterpret_cast<float2*>(sums + (warp * kInt4Rows + 16 * m + 8 * half + g) * 8 + 2 * t) = v;
          }
        asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
        for (int o = threadIdx.x; o < kInt4Rows * 8; o += kThreads) {
          const int row = o % kInt4Rows, col = o / kInt4Rows;
          if (8 * n + col >= p.M) break;
          float s = 0.0f;
#pragma unroll
          for (int v = 0; v < kWarps; ++v) s += sums[(v * kInt4Rows + row) * 8 + col];
          if (a.split > 1) {
            part[(8 * n + col) * kInt4Rows + row] = s;
          } else if (strip * kInt4Rows + row < p.N) {
            static_cast<__nv_bfloat16*>(p.out)[(8 * n + col) * p.out_stride + strip * kInt4Rows + row] =
                __float2bfloat16_rn(s);
          }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
      }
    }
  }
  if (a.split > 1) {  // one strip a cluster
    __syncthreads();
    cluster_sync();
    for (int o = rank * blockDim.x + threadIdx.x; o < p.M * kInt4Rows; o += a.split * blockDim.x) {
      const int row = o % kInt4Rows, m = o / kInt4Rows;
      float s = 0.0f;
      for (int r = 0; r < a.split; ++r) s += remote_f32(part + o, r);
      if (first * kInt4Rows + row < p.N)
        static_cast<__nv_bfloat16*>(p.out)[m * p.out_stride + first * kInt4Rows + row] = __float2bfloat16_rn(s);
    }
    cluster_sync();  // no block ends while another reads its sums
  }
}

}  // namespace

cudaError_t launch_linear_int4(const LinearInt4& p, int num_sms, cudaStream_t stream) {
  Args a{};
  a.p = p;
  a.strips = (p.N + kInt4Rows - 1) / kInt4Rows;
  if (a.p.row_strips > a.strips) a.p.row_strips = a.strips;
  a.units = (p.K + kInt4Unit - 1) / kInt4Unit;
  // Twice as many blocks while that is at most two an SM and half as many had
  // more than a stage of inputs each.  So a block may get less than a stage, and
  // the last ones none at all: they add zeros (17 units of inputs over 8
  // blocks: 3 for each of five, 2 for one, none for two).
  a.split = 1;
  while (a.split < kMostSplit && a.strips * a.split * 2 <= 2 * num_sms && a.units > a.split * kStageUnits) a.split *= 2;
  a.units_per_rank = (a.units + a.split - 1) / a.split;
  a.stage_bytes = kStageUnits * int4_record_bytes(p.group);
  a.row_offset = kStages * a.stage_bytes;
  a.row_stage_bytes = static_cast<int>(align_up(p.M * kPitch, 128));
  a.reduce_offset = a.row_offset + kRowStages * a.row_stage_bytes;
  a.part_offset = a.reduce_offset + kReduce;
  const size_t smem = a.part_offset + (a.split > 1 ? kInt4Rows * p.M * 4 : 0);
  constexpr size_t kMost = kStages * kStageUnits * int4_record_bytes(32) + kRowStages * 16 * kPitch + kReduce +
                           kInt4Rows * 16 * 4;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t err = allow(reinterpret_cast<const void*>(linear_int4_kernel), allowed, kMost, false);
  if (err != cudaSuccess) return err;
  if (a.split > 1)
    return [&] {
      cudaLaunchAttribute attr{};
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = a.split;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(a.strips * a.split);
      cfg.blockDim = dim3((kWarps + 2) * 32);
      cfg.dynamicSmemBytes = smem;
      cfg.stream = stream;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      return cudaLaunchKernelEx(&cfg, linear_int4_kernel, a);
    }();
  linear_int4_kernel<<<a.strips < 2 * num_sms ? a.strips : 2 * num_sms, (kWarps + 2) * 32, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
