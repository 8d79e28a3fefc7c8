// 4-bit weights with group scales: quantiser and packing.
//   scale = bf16(amax / 7) (1 for a group of zeros), code = 8 + w / scale
//   rounded to nearest even, within 0 .. 15; the weight is (code - 8) x scale.
#include "int4.cuh"
#include "internal.h"

namespace moe {
namespace {

// One thread a group of one output feature; neighbours read neighbours.
__global__ void __launch_bounds__(256)
quantize_kernel(const __nv_bfloat16* __restrict__ w, int64_t matrices, int64_t K, int64_t N, int group,
                uint8_t* __restrict__ codes, __nv_bfloat16* __restrict__ scales) {
  const int64_t groups = (K + group - 1) / group, total = matrices * groups * N;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t n = i % N, gi = i / N % groups, m = i / N / groups;
    const int64_t k0 = gi * group, k1 = min(K, k0 + group);
    const __nv_bfloat16* src = w + m * K * N + n;
    float amax = 0.0f;
    for (int64_t k = k0; k < k1; ++k) amax = fmaxf(amax, fabsf(__bfloat162float(src[k * N])));
    __nv_bfloat16 scale = __float2bfloat16_rn(amax / 7.0f);
    if (!(__bfloat162float(scale) > 0.0f)) scale = __float2bfloat16_rn(1.0f);
    scales[i] = scale;
    const float s = __bfloat162float(scale);
    for (int64_t k = k0; k < k1; k += 2) {
      int q[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        q[j] = min(15, max(0, 8 + __float2int_rn(__bfloat162float(src[(k + j) * N]) / s)));
      codes[(m * (K / 2) + k / 2) * N + n] = static_cast<uint8_t>(q[0] | q[1] << 4);
    }
  }
}

// One thread a word of codes (8 inputs of a row) or a scale.
__global__ void __launch_bounds__(256)
pack_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
            const uint8_t* __restrict__ up_codes, const uint16_t* __restrict__ up_scales, int64_t records, int strips,
            int units, int K, int N, int group, uint8_t* __restrict__ packed) {
  const int groups = (K + group - 1) / group, per_unit = kInt4Unit / group;
  const int bytes = int4_record_bytes(group);
  for (int64_t r = blockIdx.x; r < records; r += gridDim.x) {
    const int unit = static_cast<int>(r % units), strip = static_cast<int>(r / units % strips);
    const int64_t m = r / units / strips;
    uint8_t* dst = packed + r * bytes;
    // the feature and projection of a strip's row
    auto feature = [&](int row, bool& up) {
      up = up_codes && row >= kInt4Rows / 2;
      return up_codes ? strip * (kInt4Rows / 2) + row % (kInt4Rows / 2) : strip * kInt4Rows + row;
    };
    for (int i = threadIdx.x; i < kInt4CodeBytes / 4; i += blockDim.x) {
      const int word = i & 3, lane = i >> 2 & 31, tile = i >> 7 & 3, kb = i >> 9;
      const int row = 16 * tile + 8 * (word >> 1) + (lane >> 2);
      const int k = unit * kInt4Unit + kb * 64 + 32 * (word & 1) + 8 * (lane & 3);
      bool up;
      const int n = feature(row, up);
      uint32_t v = 0x88888888u;
      if (n < N && k < K) {
        const uint8_t* src = (up ? up_codes : codes) + (m * (K / 2) + k / 2) * static_cast<int64_t>(N) + n;
        v = 0;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t b = src[static_cast<int64_t>(p) * N];
          v |= (b & 15u) << (4 * p) | (b >> 4) << (4 * p + 16);
        }
      }
      reinterpret_cast<uint32_t*>(dst)[i] = v;
    }
    for (int i = threadIdx.x; i < per_unit * kInt4Rows; i += blockDim.x) {
      bool up;
      const int n = feature(i % kInt4Rows, up), gi = unit * per_unit + i / kInt4Rows;
      uint16_t v = 0;
      if (n < N && gi < groups) v = (up ? up_scales : scales)[(m * groups + gi) * N + n];
      reinterpret_cast<uint16_t*>(dst + kInt4CodeBytes)[i] = v;
    }
  }
}

}  // namespace

// Bytes of `matrices` matrices of N output rows (gate and up together: 2f).
size_t int4_matrix_bytes(int64_t matrices, int K, int64_t N, int group) {
  const int64_t strips = (N + kInt4Rows - 1) / kInt4Rows, units = (K + kInt4Unit - 1) / kInt4Unit;
  return static_cast<size_t>(matrices * strips * units) * int4_record_bytes(group);
}

cudaError_t launch_quantize_int4(const void* w, int64_t matrices, int64_t K, int64_t N, int group, uint8_t* codes,
                                 void* scales, int num_sms, cudaStream_t stream) {
  const int64_t total = matrices * ((K + group - 1) / group) * N;
  if (total == 0) return cudaSuccess;
  const int64_t want = (total + 255) / 256, cap = static_cast<int64_t>(num_sms) * 16;
  quantize_kernel<<<static_cast<int>(want < cap ? want : cap), 256, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(w), matrices, K, N, group, codes, static_cast<__nv_bfloat16*>(scales));
  return cudaGetLastError();
}

cudaError_t launch_pack_int4(const uint8_t* codes, const void* scales, const uint8_t* up_codes, const void* up_scales,
                             int64_t matrices, int K, int N, int group, void* packed, int num_sms,
                             cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(N) * (up_codes ? 2 : 1);
  const int strips = static_cast<int>((rows + kInt4Rows - 1) / kInt4Rows), units = (K + kInt4Unit - 1) / kInt4Unit;
  const int64_t records = matrices * strips * units, cap = static_cast<int64_t>(num_sms) * 32;
  pack_kernel<<<static_cast<int>(records < cap ? records : cap), 256, 0, stream>>>(
      codes, static_cast<const uint16_t*>(scales), up_codes, static_cast<const uint16_t*>(up_scales), records, strips,
      units, K, N, group, static_cast<uint8_t*>(packed));
  return cudaGetLastError();
}

}  // namespace moe
