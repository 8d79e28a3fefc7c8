// Launch forms of the training-step kernels.
//
// Programmatic dependent launch: a kernel that follows another on the same
// stream may be brought onto the SMs before the first one has ended.  The
// second kernel calls wait_for_previous() before it reads anything that the
// first one writes (the wait covers the whole first grid and its writes);
// the first one calls let_next_start() as early as it likes.
//
// Stealing blocks: a kernel launched with one block for each piece of work
// keeps running by cancelling launches that are still waiting and doing their
// pieces itself (cluster launch control), so pieces go to the SMs as these
// get free, without a counter in memory and without a new block's start-up.
//
// One cluster: a small problem runs as a single cluster of up to kClusterMost
// blocks that add their sums through each other's shared memory, which saves
// the second launch and its scratch (the time of a small call is the host's).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"

namespace moe {

__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

constexpr int kStealRefused = -1, kStealUnanswered = -2;

// Asks for a launch to cancel; the answer (16 bytes, in `answer`) completes the
// barrier's phase.  One thread; not again after a refusal.
__device__ __forceinline__ void steal_request(uint4* answer, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_addr(answer)),
               "r"(smem_addr(bar))
               : "memory");
}
// The x index of the block whose launch was cancelled, or kStealRefused.
__device__ __forceinline__ int steal_answer(const uint4* answer) {
  uint32_t x = 0, ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t"
      "ld.shared.b128 a, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.u32 %1, 1, 0, p;\n\t"
      "mov.u32 %0, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, a;\n\t}"
      : "=r"(x), "=r"(ok)
      : "r"(smem_addr(answer))
      : "memory");
  return ok ? static_cast<int>(x) : kStealRefused;
}

// Waits for an answer, for limit_ns at most; looks once more after that, for a
// block that was off its SM meanwhile.
__device__ __forceinline__ bool steal_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint32_t a = smem_addr(bar);
  if (mbar_try_wait(a, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  do {
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(a, parity)) return true;
  } while (global_timer_ns() - t0 <= limit_ns);
  return mbar_try_wait(a, parity);
}

// All threads of the block, each with its own limit: true in every one of them
// where the answer came to any, so that they go on alike.
__device__ __forceinline__ bool steal_told(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  return __syncthreads_or(steal_wait(bar, parity, limit_ns));
}

// All threads of the block: the index of the block whose launch was cancelled,
// kStealRefused, or kStealUnanswered after twice the limit.  A launch that was
// cancelled starts nowhere else, so an answer that some threads have not seen
// in time is waited for again and taken by all, and one that never came may
// have been a piece of work: the caller must let that be seen.
__device__ __forceinline__ int steal_next(const uint4* answer, uint64_t* bar, uint32_t parity) {
  const bool told = steal_wait(bar, parity, kWaitLimitNs);
  int block = told ? steal_answer(answer) : kStealRefused;
  if (__syncthreads_and(block >= 0)) return block;  // and all have read it
  if (!steal_told(bar, parity, kWaitLimitNs)) return kStealUnanswered;
  block = steal_answer(answer);
  __syncthreads();
  return block;
}

// What a kernel keeps of its requests: the number of answers so far, or one of
constexpr uint32_t kStealOver = ~0u, kStealLost = ~0u - 1;  // refused; unanswered

constexpr int kClusterMost = 16;  // above 8 needs the kernel's leave (allow_cluster)

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// All threads of all blocks of the cluster; writes to shared memory before it
// are visible after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Reads of another block's shared memory, at the caller's own address of it.
__device__ __forceinline__ uint32_t remote_addr(const void* own, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(own))), "r"(rank));
  return a;
}
__device__ __forceinline__ float remote_f32(const float* own, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote_addr(own, rank)) : "memory");
  return v;
}
__device__ __forceinline__ double remote_f64(const double* own, uint32_t rank) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(remote_addr(own, rank)) : "memory");
  return v;
}

// Lets the kernel have `smem` bytes of dynamic shared memory and clusters of
// kClusterMost blocks, once for each device.
inline cudaError_t allow(const void* kernel, std::atomic<uint64_t>& done, size_t smem, bool cluster) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  if (smem > 0)
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err == cudaSuccess && cluster)
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return err;
}

template <typename... Params, typename... Args>
cudaError_t launch_cluster(void (*kernel)(Params...), int blocks, int threads, size_t smem, cudaStream_t stream,
                           Args... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = blocks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             Args... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace moe
