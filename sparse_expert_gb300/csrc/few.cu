// The experts of the layer for a few tokens, the simplest form: a warp has
// one output feature of a unit and all of its tokens.
#include <cuda_fp8.h>

#include "few.cuh"
#include "int4.cuh"
#include "internal.h"

namespace moe {
namespace {

enum { kGate = 0, kUp = 1, kDown = 2 };

// Two weights of a feature, inputs 64 kb + 2 lane and the next, in fp32.
struct Weights {
  const uint8_t* packed;
  int kind, group, E, d, f, down_bn;
  size_t fp8_off[4];
  size_t int4_down;

  __device__ float2 load(int proj, int e, int n, int kb, int lane) const {
    const int K = proj == kDown ? f : d, N = proj == kDown ? d : f;
    const int nkb = K / 64;
    if (kind == MOE_WEIGHTS_BF16) {
      const int64_t base = proj == kDown ? static_cast<int64_t>(E) * 2 * d * f : 0;
      const int bn = proj == kDown ? down_bn : 128, rows = proj == kDown ? N : 2 * N;
      const int row = proj == kDown ? n : n / 64 * 128 + proj * 64 + n % 64;
      const int64_t at = base + (((static_cast<int64_t>(e) * (rows / bn) + row / bn) * nkb + kb) * bn + row % bn) * 64;
      const __nv_bfloat162 v = reinterpret_cast<const __nv_bfloat162*>(packed)[at / 2 + lane];
      return make_float2(__low2float(v), __high2float(v));
    }
    if (kind == MOE_WEIGHTS_FP8) {
      const uint8_t* codes = packed + fp8_off[proj == kDown ? 1 : 0];
      const float* scales = reinterpret_cast<const float*>(packed + fp8_off[proj == kDown ? 3 : 2]);
      const int tile = proj == kDown ? n / 128 : n / 64, tiles = proj == kDown ? N / 128 : N / 64;
      const int row = proj == kDown ? n % 128 : n % 64 / 16 * 32 + proj * 16 + n % 16;
      const uint8_t* c = codes + (((static_cast<int64_t>(e) * tiles + tile) * nkb + kb) * 128 + row) * 64 + 2 * lane;
      const int rec = proj == kDown ? kFp8DownRecord : kFp8GateUpRecord;
      const float* s = scales + ((static_cast<int64_t>(e) * (N / 128) + n / 128) * nkb + kb) * rec +
                       (proj == kUp ? 68 : 0) + 2 * lane;
      float v[2];
      for (int i = 0; i < 2; ++i) v[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(c[i], __NV_E4M3))) * s[i];
      return make_float2(v[0], v[1]);
    }
    const int units = K / kInt4Unit, unit = kb / 2;
    const int strip = proj == kDown ? n / 64 : n / 32, strips = proj == kDown ? N / 64 : N / 32;
    const int row = proj == kDown ? n % 64 : n % 32 + 32 * proj;
    const uint8_t* r = packed + (proj == kDown ? int4_down : 0) +
                       ((static_cast<int64_t>(e) * strips + strip) * units + unit) * int4_record_bytes(group);
    const int k = 2 * lane, l = (row % 8) * 4 + k % 32 / 8, word = (row % 16) / 8 * 2 + k / 32;
    const uint32_t w = reinterpret_cast<const uint32_t*>(r)[(((kb % 2) * 4 + row / 16) * 32 + l) * 4 + word];
    const int p = k % 8 / 2;
    const float s = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(
        r + kInt4CodeBytes)[(kb % 2 * 64 + k) / group * kInt4Rows + row]);
    return make_float2(s * (static_cast<int>(w >> (4 * p) & 15) - 8), s * (static_cast<int>(w >> (4 * p + 16) & 15) - 8));
  }
};

__device__ float2 row_pair(const __nv_bfloat16* rows, int64_t width, int row, int k) {
  const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(rows + row * width + k);
  return make_float2(__low2float(v), __high2float(v));
}

__device__ float warp_sum(float v) {
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

__global__ void __launch_bounds__(256) gate_up_kernel(const FewExperts p, const Weights w) {
  const int lane = threadIdx.x & 31, n = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (static_cast<int>(blockIdx.y) >= p.header->n_units || n >= p.f) return;
  const FewUnit u = p.units[blockIdx.y];
  float g[kFewChunk] = {}, v[kFewChunk] = {};
  for (int kb = 0; kb < p.d / 64; ++kb) {
    const float2 wg = w.load(kGate, u.expert, n, kb, lane), wu = w.load(kUp, u.expert, n, kb, lane);
    uint64_t rest = u.tokens;
#pragma unroll
    for (int i = 0; i < kFewChunk; ++i)
      if (rest) {
        const float2 x = row_pair(static_cast<const __nv_bfloat16*>(p.x), p.d, __ffsll(rest) - 1, kb * 64 + 2 * lane);
        rest &= rest - 1;
        g[i] += wg.x * x.x + wg.y * x.y;
        v[i] += wu.x * x.x + wu.y * x.y;
      }
  }
#pragma unroll
  for (int i = 0; i < kFewChunk; ++i) {
    const float a = warp_sum(g[i]), b = warp_sum(v[i]);
    if (lane == 0 && i < __popcll(u.tokens))
      static_cast<__nv_bfloat16*>(p.h)[static_cast<int64_t>(u.row + i) * p.f + n] =
          __float2bfloat16_rn(a / (1.0f + __expf(-a)) * b);
  }
}

__global__ void __launch_bounds__(256) down_kernel(const FewExperts p, const Weights w) {
  const int lane = threadIdx.x & 31, n = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (static_cast<int>(blockIdx.y) >= p.header->n_units || n >= p.d) return;
  const FewUnit u = p.units[blockIdx.y];
  float y[kFewChunk] = {};
  const int rows = __popcll(u.tokens);
  for (int kb = 0; kb < p.f / 64; ++kb) {
    const float2 wd = w.load(kDown, u.expert, n, kb, lane);
#pragma unroll
    for (int i = 0; i < kFewChunk; ++i)
      if (i < rows) {
        const float2 h = row_pair(static_cast<const __nv_bfloat16*>(p.h), p.f, u.row + i, kb * 64 + 2 * lane);
        y[i] += wd.x * h.x + wd.y * h.y;
      }
  }
#pragma unroll
  for (int i = 0; i < kFewChunk; ++i) {
    const float a = warp_sum(y[i]);
    if (lane == 0 && i < rows) p.y[static_cast<int64_t>(u.row + i) * p.d + n] = a;
  }
}

__global__ void __launch_bounds__(256) combine_kernel(const FewExperts p) {
  const int t = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x;
  if (n >= p.d) return;
  float s = 0.0f;
  for (int j = 0; j < p.k; ++j)
    s += p.topk_w[t * p.k + j] * p.y[static_cast<int64_t>(p.pair_row[t * p.k + j]) * p.d + n];
  static_cast<__nv_bfloat16*>(p.out)[static_cast<int64_t>(t) * p.d + n] = __float2bfloat16_rn(s);
}

}  // namespace

cudaError_t launch_few_experts(const FewExperts& p, int num_sms, cudaStream_t stream) {
  Weights w{static_cast<const uint8_t*>(p.packed), p.weights, p.group, p.E, p.d, p.f, down_tile_n(p.d), {}, 0};
  if (p.weights == MOE_WEIGHTS_FP8) fp8_packed_bytes(p.E, p.d, p.f, w.fp8_off);
  if (p.weights == MOE_WEIGHTS_INT4) w.int4_down = align_up(int4_matrix_bytes(p.E, p.d, 2 * p.f, p.group));
  const int units = p.T * p.k;
  gate_up_kernel<<<dim3(p.f / 8, units), 256, 0, stream>>>(p, w);
  down_kernel<<<dim3(p.d / 8, units), 256, 0, stream>>>(p, w);
  combine_kernel<<<dim3((p.d + 255) / 256, p.T), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
