// Products of a few rows with 4-bit weights, the simplest form: a warp has
// one output feature and all rows.
#include "int4.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kMost = 16;

__global__ void __launch_bounds__(256) linear_int4_kernel(const LinearInt4 p) {
  const int lane = threadIdx.x & 31, n = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (n >= p.N) return;
  const int units = (p.K + kInt4Unit - 1) / kInt4Unit, row = n % kInt4Rows;
  float y[kMost] = {};
  for (int unit = 0; unit < units; ++unit) {
    const uint8_t* r = static_cast<const uint8_t*>(p.packed) +
                       (static_cast<int64_t>(n / kInt4Rows) * units + unit) * int4_record_bytes(p.group);
    for (int k = 2 * lane; k < kInt4Unit; k += 64) {
      if (unit * kInt4Unit + k >= p.K) break;
      const int l = (row % 8) * 4 + k % 32 / 8, word = (row % 16) / 8 * 2 + k % 64 / 32, pos = k % 8 / 2;
      const uint32_t w = reinterpret_cast<const uint32_t*>(r)[((k / 64 * 4 + row / 16) * 32 + l) * 4 + word];
      const float s = __bfloat162float(
          reinterpret_cast<const __nv_bfloat16*>(r + kInt4CodeBytes)[k / p.group * kInt4Rows + row]);
      const float w0 = s * (static_cast<int>(w >> (4 * pos) & 15) - 8);
      const float w1 = s * (static_cast<int>(w >> (4 * pos + 16) & 15) - 8);
#pragma unroll
      for (int m = 0; m < kMost; ++m)
        if (m < p.M) {
          const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(
              static_cast<const __nv_bfloat16*>(p.x) + m * p.x_stride + unit * kInt4Unit + k);
          y[m] += w0 * __low2float(x) + w1 * __high2float(x);
        }
    }
  }
#pragma unroll
  for (int m = 0; m < kMost; ++m) {
    float a = y[m];
    for (int s = 16; s > 0; s >>= 1) a += __shfl_xor_sync(0xffffffffu, a, s);
    if (lane == 0 && m < p.M)
      static_cast<__nv_bfloat16*>(p.out)[m * p.out_stride + n] = __float2bfloat16_rn(a);
  }
}

}  // namespace

cudaError_t launch_linear_int4(const LinearInt4& p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  linear_int4_kernel<<<(p.N + 7) / 8, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
