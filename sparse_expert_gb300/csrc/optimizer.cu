// AdamW over a list of tensors, and the norm of a list of gradients.
//
//   g = grad * factor;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = p - (lr wd p + lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps))
//
// The list travels in the kernel's parameters (up to 32 KB), so a call is one
// launch per kCapacity tensors, needs no copy to the device, keeps nothing
// from call to call and can be captured into a graph.  The tensors are cut
// into chunks of kChunkValues values; chunks are numbered through the list,
// and a block finds its tensor by bisection of the first chunk numbers.
//
// 8-bit states: m and sqrt(v) as E4M3 codes with one fp32 scale per 128
// values.  sqrt(v) and not v: E4M3 spans a ratio of 2^18 (to a sixteenth of
// the value or better above 2^-15 of the maximum), which as v itself is 2^36.
// The products and sums of m and v are rounded one by one (no fused
// multiply-add), so that the codes do not depend on how they are contracted.
//
// Bound by memory with 32-bit states (403M bf16 weights with masters 1589 us =
// 7.1 TB/s) and with 8-bit states and masters (528M: 1248 us = 6.8 TB/s); with
// 8-bit states alone, 62 instructions a value bind it, in 85 % of the issue
// slots (202M: 392 us = 5.2 TB/s).  Some of them are spills: the kernel for
// 8-bit states holds all forms of a chunk in 40 registers, and its threads
// store 212 and load 308 bytes of them in the worst case.
#include <cuda_fp8.h>

#include "common.cuh"
#include "elem.cuh"
#include "internal.h"
#include "launch.cuh"

namespace moe {
namespace {

constexpr int kBlockThreads = 256;
constexpr int kScaleBlock = 128;
constexpr int kChunkValues = kBlockThreads * 8;  // one vector a thread
static_assert(kChunkValues == kAdamWChunk, "the largest tensor's chunks have numbers");
// of the gradient norm:
constexpr int kNormVectors = 4;        // 32-byte vectors a thread of a chunk
static_assert(kNormVectors * kBlockThreads * 8 >= kAdamWChunk, "and so have its larger chunks here");
constexpr int kLongShare = 24;         // chunks a resident block beyond which there are more blocks
constexpr int kClusterThreads = 1024;  // of a block of the one cluster for small lists,
constexpr int kClusterRounds = 2;      // and its chunks a block
constexpr float kE4M3Max = 448.0f;
constexpr float kTinyBlock = 7.888609052210118e-31f;  // 2^-100

struct Tensor {
  void* param;
  float* master;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  float decay;
  uint8_t param_type, grad_type, bits8, vec;  // vec: vectors lie at their alignment
};

template <int kCapacity>
struct List {
  int count;
  int chunks;
  moe_adamw_hyper_t hyper;
  const moe_adamw_hyper_t* hyper_dev;
  const float* grad_scale;
  int first[kCapacity + 1];  // number of each tensor's first chunk
  Tensor t[kCapacity];
};

// The tensor of a chunk: the last one whose first chunk is not after it
// (tensors without values are not in the list).
template <int kCapacity>
__device__ __forceinline__ int tensor_of(const List<kCapacity>& list, int chunk) {
  int lo = 0, hi = list.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (list.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float load_any(const void* p, int type, int64_t i) {
  if (type == MOE_F32) return static_cast<const float*>(p)[i];
  if (type == MOE_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
  return to_f32(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ void store_any(void* p, int type, int64_t i, float v) {
  if (type == MOE_F32) static_cast<float*>(p)[i] = v;
  else if (type == MOE_BF16) static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(v);
  else static_cast<__half*>(p)[i] = from_f32<__half>(v);
}

// Eight values of a thread: 32 bytes of fp32 in one access, 16 bytes of a
// 16-bit type, kept as they are until every load of the thread is on its way.
struct Raw8 {
  uint32_t w[8];
};

__device__ __forceinline__ void load8_f32(const float* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}

__device__ __forceinline__ void load8(const void* p, int type, int64_t i, Raw8& r) {
  if (type == MOE_F32) {
    load8_f32(static_cast<const float*>(p) + i, r.w);
  } else {
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "l"(static_cast<const uint16_t*>(p) + i));
  }
}

// The first `count` values (of `size` bytes) of the eight, one by one; the
// rest of the words stays as it is.
__device__ __forceinline__ void load_some(const void* p, int size, int64_t j, int count, uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= count) continue;
    if (size == 4) w[i] = static_cast<const uint32_t*>(p)[j + i];
    else if (size == 2) w[i / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[j + i]) << (16 * (i & 1));
    else w[i / 4] |= static_cast<uint32_t>(static_cast<const uint8_t*>(p)[j + i]) << (8 * (i & 3));
  }
}

__device__ __forceinline__ void values8(const Raw8& r, int type, float2 (&v)[4]) {
  if (type == MOE_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
  } else {
    const uint4 u = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    if (type == MOE_BF16) unpack_pairs<__nv_bfloat16>(u, v);
    else unpack_pairs<__half>(u, v);
  }
}

__device__ __forceinline__ void store8(void* p, int type, int64_t i, const float2 (&v)[4]) {
  if (type == MOE_F32) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<float*>(p) + i),
                 "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y)
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        type == MOE_BF16 ? pack_pairs<__nv_bfloat16>(v) : pack_pairs<__half>(v);
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The largest of a and the magnitudes of b and c.
__device__ __forceinline__ float max3_nan_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float decode(uint8_t code, float scale) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(code, __NV_E4M3);
  return __fmul_rn(__half2float(__half(h)), scale);
}

// The scale of a block with maximum `amax`, and the factor into the codes.
__device__ __forceinline__ void block_scale(float amax, float* scale, float* inv) {
  const bool tiny = amax < kTinyBlock;  // not for NaN: it spreads to the block
  *scale = tiny ? 1.0f : __fmul_rn(amax, 1.0f / kE4M3Max);
  *inv = tiny ? 1.0f : __fdiv_rn(kE4M3Max, amax);
}

// A quotient for the update, which goes into a sum that rounds away far more
// than its two ulps.  Denormal arguments count as zero: a root of a positive
// second moment is above 1e-23.
__device__ __forceinline__ float divide_approx(float a, float b) {
  float r;
  asm("div.approx.ftz.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The sum of two products rounded on their own: as single additions, because
// the assembler merges a packed addition with the packed product before it.
__device__ __forceinline__ float2 add_single(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// The new moments (products and sums rounded singly), the root of the second
// and the new parameter of two values.
__device__ __forceinline__ void adamw_pair(const moe_adamw_hyper_t& h, float decay, float2 g, float2& p, float2& m,
                                           float2& v, float2& root) {
  m = add_single(mul2(m, both(h.beta1)), mul2(g, both(h.one_minus_beta1)));
  v = add_single(mul2(v, both(h.beta2)), mul2(mul2(g, g), both(h.one_minus_beta2)));
  root = make_float2(__fsqrt_rn(v.x), __fsqrt_rn(v.y));
  const float2 denom = fma2(root, both(h.inv_sqrt_bias), both(h.eps));
  const float2 num = mul2(m, both(h.step_size));
  const float2 update = make_float2(divide_approx(num.x, denom.x), divide_approx(num.y, denom.y));
  const float2 change = fma2(p, both(decay), update);
  p = fma2(change, both(-1.0f), p);
}

// Not zero if a byte of w is zero.
__device__ __forceinline__ uint32_t has_zero_byte(uint32_t w) { return (w - 0x01010101u) & ~w & 0x80808080u; }

// E4M3 codes of eight values, four to a word.
__device__ __forceinline__ uint2 encode8(const float2 (&x)[4], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __nv_cvt_float2_to_fp8x2(mul2(x[i], both(inv)), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

__device__ __forceinline__ void decode8(const uint2& codes, float scale, float2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t word = i < 2 ? codes.x : codes.y;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<uint16_t>(word >> (16 * (i & 1))), __NV_E4M3);
    v[i] = mul2(__half22float2(__half2(h)), both(scale));
  }
}

// A whole chunk of a tensor with aligned pointers: eight consecutive values
// a thread, so sixteen lanes hold the 128 values of a scale.
template <bool kBits8>
__device__ __forceinline__ void adamw_whole_chunk(const Tensor& t, const moe_adamw_hyper_t& h, const float* factor_p,
                                            int64_t begin) {
  const int64_t j = begin + threadIdx.x * 8;
  Raw8 raw_g, raw_p, raw_m, raw_v;
  uint2 code_m, code_v;
  float ms, vs;
  load8(t.grad, t.grad_type, j, raw_g);
  const bool master = t.master != nullptr;
  const int p_type = master ? static_cast<int>(MOE_F32) : t.param_type;
  load8(master ? t.master : t.param, p_type, j, raw_p);
  if (kBits8) {
    code_m = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + j);
    code_v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + j);
    ms = t.m_scale[j / kScaleBlock];
    vs = t.v_scale[j / kScaleBlock];
  } else {
    load8_f32(static_cast<const float*>(t.m) + j, raw_m.w);
    load8_f32(static_cast<const float*>(t.v) + j, raw_v.w);
  }
  const float factor = factor_p ? *factor_p : 1.0f;
  if (!isfinite(factor)) return;
  const float decay = h.decay * t.decay;
  float2 g[4], p[4], m[4], v[4], root[4];
  values8(raw_g, t.grad_type, g);
  values8(raw_p, p_type, p);
  if (kBits8) {
    decode8(code_m, ms, m);
    decode8(code_v, vs, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], v[i]);
  } else {
    values8(raw_m, MOE_F32, m);
    values8(raw_v, MOE_F32, v);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) adamw_pair(h, decay, mul2(g[i], both(factor)), p[i], m[i], v[i], root[i]);
  if (master) store8(t.master, MOE_F32, j, p);
  store8(t.param, t.param_type, j, p);
  if (!kBits8) {
    store8(t.m, MOE_F32, j, m);
    store8(t.v, MOE_F32, j, v);
    return;
  }
  float m_max = 0.0f, v_max = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m_max = max3_nan_abs(m_max, m[i].x, m[i].y);
    v_max = max3_nan_abs(v_max, root[i].x, root[i].y);
  }
#pragma unroll
  for (int s = 8; s > 0; s >>= 1) {
    m_max = max_nan(m_max, __shfl_xor_sync(0xffffffffu, m_max, s));
    v_max = max_nan(v_max, __shfl_xor_sync(0xffffffffu, v_max, s));
  }
  float m_scale, m_inv, v_scale, v_inv;
  block_scale(m_max, &m_scale, &m_inv);
  block_scale(v_max, &v_scale, &v_inv);
  *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + j) = encode8(m, m_inv);
  uint2 codes = encode8(root, v_inv);
  if (has_zero_byte(codes.x) | has_zero_byte(codes.y)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& w = i < 4 ? codes.x : codes.y;
      const uint32_t one = 1u << (8 * (i & 3));
      if ((w & (one * 255u)) == 0 && (i & 1 ? root[i / 2].y : root[i / 2].x) > 0.0f) w |= one;
    }
  }
  *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + j) = codes;
  if ((threadIdx.x & 15) == 0) {
    t.m_scale[j / kScaleBlock] = m_scale;
    t.v_scale[j / kScaleBlock] = v_scale;
  }
}

// The last, partial chunk of such a tensor: the thread at the tensor's end
// reads and writes its values one by one, those behind it none (their values
// are zero and raise no maximum).
struct Loaded {
  Raw8 g, p, m, v;  // m, v: with 8 bits the codes, in the first two words
  float ms, vs;
  int count;        // values of the eight that exist
};

template <bool kBits8>
__device__ __forceinline__ void load_vectors(const Tensor& t, int64_t j, Loaded& x) {
  const bool master = t.master != nullptr;
  const int p_type = master ? static_cast<int>(MOE_F32) : t.param_type;
  const void* p_in = master ? t.master : t.param;
  x.ms = x.vs = 0.0f;
  x.count = 8;
  if (j + 8 <= t.n) {
    load8(t.grad, t.grad_type, j, x.g);
    load8(p_in, p_type, j, x.p);
    if (kBits8) {
      const uint2 m = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + j);
      const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + j);
      x.m.w[0] = m.x, x.m.w[1] = m.y, x.v.w[0] = v.x, x.v.w[1] = v.y;
    } else {
      load8_f32(static_cast<const float*>(t.m) + j, x.m.w);
      load8_f32(static_cast<const float*>(t.v) + j, x.v.w);
    }
  } else {
    x.count = t.n > j ? static_cast<int>(t.n - j) : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.g.w[i] = x.p.w[i] = x.m.w[i] = x.v.w[i] = 0;
    load_some(t.grad, t.grad_type == MOE_F32 ? 4 : 2, j, x.count, x.g.w);
    load_some(p_in, p_type == MOE_F32 ? 4 : 2, j, x.count, x.p.w);
    load_some(t.m, kBits8 ? 1 : 4, j, x.count, x.m.w);
    load_some(t.v, kBits8 ? 1 : 4, j, x.count, x.v.w);
  }
  if (kBits8 && x.count > 0) {
    x.ms = t.m_scale[j / kScaleBlock];
    x.vs = t.v_scale[j / kScaleBlock];
  }
}

template <bool kBits8>
__device__ __forceinline__ void step_vectors(const Tensor& t, const moe_adamw_hyper_t& h, float factor, int64_t j,
                                             const Loaded& x) {
  const bool master = t.master != nullptr;
  const float decay = h.decay * t.decay;
  float2 g[4], p[4], m[4], v[4], root[4];
  values8(x.g, t.grad_type, g);
  values8(x.p, master ? static_cast<int>(MOE_F32) : t.param_type, p);
  if (kBits8) {
    decode8(make_uint2(x.m.w[0], x.m.w[1]), x.ms, m);
    decode8(make_uint2(x.v.w[0], x.v.w[1]), x.vs, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], v[i]);
  } else {
    values8(x.m, MOE_F32, m);
    values8(x.v, MOE_F32, v);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) adamw_pair(h, decay, mul2(g[i], both(factor)), p[i], m[i], v[i], root[i]);
  if (x.count == 8) {
    if (master) store8(t.master, MOE_F32, j, p);
    store8(t.param, t.param_type, j, p);
    if (!kBits8) {
      store8(t.m, MOE_F32, j, m);
      store8(t.v, MOE_F32, j, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= x.count) continue;
      const float pi = i & 1 ? p[i / 2].y : p[i / 2].x;
      if (master) t.master[j + i] = pi;
      store_any(t.param, t.param_type, j + i, pi);
      if (!kBits8) {
        static_cast<float*>(t.m)[j + i] = i & 1 ? m[i / 2].y : m[i / 2].x;
        static_cast<float*>(t.v)[j + i] = i & 1 ? v[i / 2].y : v[i / 2].x;
      }
    }
  }
  if (!kBits8) return;
  float m_max = 0.0f, v_max = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m_max = max3_nan_abs(m_max, m[i].x, m[i].y);
    v_max = max3_nan_abs(v_max, root[i].x, root[i].y);
  }
  // the first exchange leaves lanes 0-7 of the sixteen with maxima of m and
  // lanes 8-15 with those of the roots; each half makes its scale and hands
  // the other half a copy
  const bool upper = threadIdx.x & 8;
  float top = max_nan(upper ? v_max : m_max, __shfl_xor_sync(0xffffffffu, upper ? m_max : v_max, 8));
#pragma unroll
  for (int s = 4; s > 0; s >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, s));
  float scale, inv;
  block_scale(top, &scale, &inv);
  const float other = __shfl_xor_sync(0xffffffffu, inv, 8);
  const uint2 m_codes = encode8(m, upper ? other : inv);
  uint2 codes = encode8(root, upper ? inv : other);
  if (has_zero_byte(codes.x) | has_zero_byte(codes.y)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& w = i < 4 ? codes.x : codes.y;
      const uint32_t one = 1u << (8 * (i & 3));
      if ((w & (one * 255u)) == 0 && (i & 1 ? root[i / 2].y : root[i / 2].x) > 0.0f) w |= one;
    }
  }
  if (x.count == 8) {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + j) = m_codes;
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + j) = codes;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= x.count) continue;
      static_cast<uint8_t*>(t.m)[j + i] = static_cast<uint8_t>((i < 4 ? m_codes.x : m_codes.y) >> (8 * (i & 3)));
      static_cast<uint8_t*>(t.v)[j + i] = static_cast<uint8_t>((i < 4 ? codes.x : codes.y) >> (8 * (i & 3)));
    }
  }
  // lane 0 of the sixteen writes m's scale, lane 8 the roots' (their block
  // exists where its first value does)
  const int64_t block = j / kScaleBlock;
  if ((threadIdx.x & 7) == 0 && block * kScaleBlock < t.n) (upper ? t.v_scale : t.m_scale)[block] = scale;
}

template <bool kBits8>
__device__ __forceinline__ void adamw_last_chunk(const Tensor& t, const moe_adamw_hyper_t& h, const float* factor_p,
                                                 int64_t begin) {
  const int64_t j = begin + threadIdx.x * 8;
  Loaded x;
  load_vectors<kBits8>(t, j, x);
  const float factor = factor_p ? *factor_p : 1.0f;
  if (!isfinite(factor)) return;
  step_vectors<kBits8>(t, h, factor, j, x);
}

// A chunk of a tensor whose pointers are not all at 32-byte boundaries: a warp
// takes blocks of 128 values, lane + 32 i of each, in accesses of one value.
// Tensors with allocations of their own never come here.  Bound by the number
// of its accesses (50M bf16 weights with masters: 451 us where vectors take
// 204, with 8-bit states 406 and 123).
__device__ __forceinline__ void adamw_scalar_chunk(const Tensor& t, const moe_adamw_hyper_t& h, const float* factor_p,
                                                   int64_t begin) {
  const float factor = factor_p ? *factor_p : 1.0f;
  if (!isfinite(factor)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float decay = h.decay * t.decay;
  for (int64_t b0 = begin + warp * kScaleBlock; b0 < t.n && b0 < begin + kChunkValues;
       b0 += kScaleBlock * (kBlockThreads / 32)) {
    const int64_t block = b0 / kScaleBlock;
    const float ms = t.bits8 ? t.m_scale[block] : 1.0f, vs = t.bits8 ? t.v_scale[block] : 1.0f;
    float m[4], root[4];
    float m_max = 0.0f, v_max = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t j = b0 + lane + 32 * i;
      m[i] = root[i] = 0.0f;
      if (j >= t.n) continue;
      const float g = __fmul_rn(load_any(t.grad, t.grad_type, j), factor);
      float p = t.master ? t.master[j] : load_any(t.param, t.param_type, j);
      float v;
      if (t.bits8) {
        m[i] = decode(static_cast<const uint8_t*>(t.m)[j], ms);
        v = decode(static_cast<const uint8_t*>(t.v)[j], vs);
        v = __fmul_rn(v, v);
      } else {
        m[i] = static_cast<const float*>(t.m)[j];
        v = static_cast<const float*>(t.v)[j];
      }
      float2 p2 = both(p), m2 = both(m[i]), v2 = both(v), root2;
      adamw_pair(h, decay, both(g), p2, m2, v2, root2);
      p = p2.x, m[i] = m2.x, v = v2.x, root[i] = root2.x;
      if (t.master) t.master[j] = p;
      store_any(t.param, t.param_type, j, p);
      if (!t.bits8) {
        static_cast<float*>(t.m)[j] = m[i];
        static_cast<float*>(t.v)[j] = v;
      }
      m_max = max_nan(m_max, fabsf(m[i]));
      v_max = max_nan(v_max, root[i]);
    }
    if (!t.bits8) continue;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      m_max = max_nan(m_max, __shfl_xor_sync(0xffffffffu, m_max, s));
      v_max = max_nan(v_max, __shfl_xor_sync(0xffffffffu, v_max, s));
    }
    float m_scale, m_inv, v_scale, v_inv;
    block_scale(m_max, &m_scale, &m_inv);
    block_scale(v_max, &v_scale, &v_inv);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t j = b0 + lane + 32 * i;
      if (j >= t.n) continue;
      static_cast<uint8_t*>(t.m)[j] = __nv_cvt_float_to_fp8(__fmul_rn(m[i], m_inv), __NV_SATFINITE, __NV_E4M3);
      uint8_t code = __nv_cvt_float_to_fp8(__fmul_rn(root[i], v_inv), __NV_SATFINITE, __NV_E4M3);
      if (code == 0 && root[i] > 0.0f) code = 1;
      static_cast<uint8_t*>(t.v)[j] = code;
    }
    if (lane == 0) {
      t.m_scale[block] = m_scale;
      t.v_scale[block] = v_scale;
    }
  }
}

// kBits8: some tensor of the list has 8-bit states.  Those steps are bound by
// the latency of their small loads and take 6 blocks an SM (40 registers):
// 202M bf16 weights without masters 392 us against 462 with 5 blocks; steps
// with 32-bit states are bound by memory and faster with 5 (201M weights with
// masters 798 us, 856 with 6).
template <int kCapacity, bool kBits8>
__global__ void __launch_bounds__(kBlockThreads, kBits8 ? 6 : 5)
    adamw_kernel(const __grid_constant__ List<kCapacity> list) {
  const moe_adamw_hyper_t h = list.hyper_dev ? *list.hyper_dev : list.hyper;
  const int which = tensor_of(list, blockIdx.x);
  const Tensor& t = list.t[which];
  const int64_t begin = static_cast<int64_t>(blockIdx.x - list.first[which]) * kChunkValues;
  const bool whole = begin + kChunkValues <= t.n;
  if (!t.vec) {
    adamw_scalar_chunk(t, h, list.grad_scale, begin);
  } else if (kBits8 && t.bits8) {
    if (whole) adamw_whole_chunk<true>(t, h, list.grad_scale, begin);
    else adamw_last_chunk<true>(t, h, list.grad_scale, begin);
  } else {
    if (whole) adamw_whole_chunk<false>(t, h, list.grad_scale, begin);
    else adamw_last_chunk<false>(t, h, list.grad_scale, begin);
  }
}

// ---- gradient norm
// Sum over the block in a fixed order, in thread 0.
__device__ double block_sum(double v, double* red) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double total = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) total += red[i];
  return total;
}

__device__ __forceinline__ void write_norm(double squares, float max_norm, float* out) {
  const double norm = sqrt(squares);
  out[0] = static_cast<float>(norm);
  out[1] = !isfinite(out[0]) ? nanf("") : norm > max_norm ? static_cast<float>(max_norm / norm) : 1.0f;
}

// The squares of all gradients: one reading of them, bound by memory. A block
// takes chunks blockIdx.x, + gridDim.x, ... of kNormVectors 32-byte vectors a
// thread, all loads of a chunk in flight before its first use; the vectors of
// a tensor start at its first 32-byte boundary, and the values before it go
// with the first chunk. Up to kLongShare chunks a resident block, the blocks
// are those that the SMs hold at once (62M bf16 values 23.4 us); beyond, they
// are as many as there is room for partial sums, taken by the SMs as they get
// free (403M bf16 values 115 us = 7.0 TB/s, with resident blocks alone 120).
// A thread adds in fp32, threads and blocks in fp64, in a fixed order. As one
// cluster (`out` given), its first block writes the result.
template <int kCapacity, int kThreads>
__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ List<kCapacity> list,
                                                           double* __restrict__ partial, float max_norm, float* out) {
  __shared__ double red[kThreads / 32], block_squares;
  let_next_start();
  float2 s[4] = {both(0.0f), both(0.0f), both(0.0f), both(0.0f)};
  float odd = 0.0f;
  for (int chunk = blockIdx.x; chunk < list.chunks; chunk += gridDim.x) {
    const int which = tensor_of(list, chunk);
    const Tensor& t = list.t[which];
    const int esize = t.grad_type == MOE_F32 ? 4 : 2, per = 32 / esize;
    const int64_t head = static_cast<int64_t>((32 - (reinterpret_cast<uintptr_t>(t.grad) & 31)) & 31) / esize;
    const int64_t begin = head + static_cast<int64_t>(chunk - list.first[which]) * (kNormVectors * kThreads * per);
    uint32_t raw[kNormVectors][8];
    const int64_t left = t.n - begin;  // values from the chunk's begin
#pragma unroll
    for (int i = 0; i < kNormVectors; ++i) {
      const int at = (i * kThreads + threadIdx.x) * per;
      if (at + per <= left)
        load8_f32(reinterpret_cast<const float*>(static_cast<const char*>(t.grad) + (begin + at) * esize), raw[i]);
      else
#pragma unroll
        for (int k = 0; k < 8; ++k) raw[i][k] = 0;
    }
#pragma unroll
    for (int i = 0; i < kNormVectors; ++i) {
      if (t.grad_type == MOE_F32) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 g = make_float2(__uint_as_float(raw[i][2 * k]), __uint_as_float(raw[i][2 * k + 1]));
          s[k] = fma2(g, g, s[k]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float f[2];
          if (t.grad_type == MOE_BF16) Word<__nv_bfloat16>::unpack(raw[i][k], f);
          else Word<__half>::unpack(raw[i][k], f);
          const float2 g = make_float2(f[0], f[1]);
          s[k & 3] = fma2(g, g, s[k & 3]);
        }
      }
    }
    // the values before the first vector, and those after the last whole one
    if (chunk == list.first[which] && threadIdx.x < head && threadIdx.x < t.n) {
      const float g = load_any(t.grad, t.grad_type, threadIdx.x);
      odd += g * g;
    }
    if (left > 0 && left < kNormVectors * kThreads * per && threadIdx.x < left % per) {
      const float g = load_any(t.grad, t.grad_type, t.n - 1 - threadIdx.x);
      odd += g * g;
    }
  }
  const float2 all = add2(add2(s[0], s[1]), add2(s[2], s[3]));
  const double total = block_sum(all.x + all.y + odd, red);
  if (!out) {
    if (threadIdx.x == 0) partial[blockIdx.x] = total;
    return;
  }
  if (threadIdx.x == 0) block_squares = total;
  cluster_sync();
  if (cluster_rank() == 0 && threadIdx.x == 0) {
    double squares = 0.0;
    for (uint32_t k = 0; k < gridDim.x; ++k) squares += remote_f64(&block_squares, k);
    write_norm(squares, max_norm, out);
  }
  cluster_sync();  // no block leaves while another reads its sum
}

// The norm from the blocks' sums, in one block and a fixed order: latency only
// (launched while the squares are summed, about 3 us behind them).
__global__ void __launch_bounds__(kBlockThreads) norm_kernel(const double* __restrict__ partial, int blocks,
                                                             float max_norm, float* __restrict__ out) {
  __shared__ double red[kBlockThreads / 32];
  wait_for_previous();
  double s = 0.0;
  for (int b = threadIdx.x; b < blocks; b += kBlockThreads) s += partial[b];
  s = block_sum(s, red);
  if (threadIdx.x == 0) write_norm(s, max_norm, out);
}

// ---- lists
bool all_aligned(const moe_adamw_tensor_t& s) {
  uintptr_t low = reinterpret_cast<uintptr_t>(s.param) | reinterpret_cast<uintptr_t>(s.master) |
                  reinterpret_cast<uintptr_t>(s.grad) | reinterpret_cast<uintptr_t>(s.m) |
                  reinterpret_cast<uintptr_t>(s.v);
  return low % 32 == 0;
}

template <int kCapacity>
int fill(List<kCapacity>& list, const moe_adamw_tensor_t* tensors, int n_tensors, int norm_threads, int* at) {
  list.count = 0;
  int64_t chunks = 0;
  while (*at < n_tensors && list.count < kCapacity) {
    const moe_adamw_tensor_t& s = tensors[*at];
    const int chunk =
        norm_threads == 0 ? kChunkValues : kNormVectors * norm_threads * 32 / (s.grad_type == MOE_F32 ? 4 : 2);
    const int64_t more = (s.n + chunk - 1) / chunk;
    if (chunks + more > INT32_MAX) break;  // not at the list's first: kTensorMaxValues
    ++*at;
    if (s.n == 0) continue;
    list.first[list.count] = static_cast<int>(chunks);
    list.t[list.count++] = Tensor{s.param, s.master, s.grad, s.m, s.v, s.m_scale, s.v_scale, s.n, s.decay,
                                  static_cast<uint8_t>(s.param_type), static_cast<uint8_t>(s.grad_type),
                                  static_cast<uint8_t>(s.state_bits == 8), static_cast<uint8_t>(all_aligned(s))};
    chunks += more;
  }
  list.chunks = static_cast<int>(chunks);
  return list.chunks;
}

template <int kCapacity>
cudaError_t adamw_all(const moe_adamw_tensor_t* tensors, int n_tensors, const moe_adamw_hyper_t* hyper,
                      const moe_adamw_hyper_t* hyper_dev, const float* grad_scale, cudaStream_t stream) {
  List<kCapacity> list;
  if (hyper) list.hyper = *hyper;
  list.hyper_dev = hyper_dev;
  list.grad_scale = grad_scale;
  for (int at = 0; at < n_tensors;) {
    if (fill(list, tensors, n_tensors, 0, &at) == 0) continue;
    bool bits8 = false;
    for (int i = 0; i < list.count; ++i) bits8 |= list.t[i].bits8 != 0;
    if (bits8) adamw_kernel<kCapacity, true><<<list.chunks, kBlockThreads, 0, stream>>>(list);
    else adamw_kernel<kCapacity, false><<<list.chunks, kBlockThreads, 0, stream>>>(list);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

template <int kCapacity>
cudaError_t norm_all(const moe_adamw_tensor_t* tensors, int n_tensors, float max_norm, float* out, double* partial,
                     int num_sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  List<kCapacity> list{};
  const int launches = (n_tensors + kCapacity - 1) / kCapacity;
  const int most = launches > 0 ? kGradNormMaxBlocks / launches : 1;
  if (most < 1) return cudaErrorInvalidValue;
  int blocks = 0;
  if (launches == 1) {
    int at = 0;
    const int chunks = fill(list, tensors, n_tensors, kClusterThreads, &at);
    if (at == n_tensors && chunks <= kClusterMost * kClusterRounds) {
      auto kernel = squares_kernel<kCapacity, kClusterThreads>;
      const cudaError_t err = allow(reinterpret_cast<const void*>(kernel), done, 0, true);
      if (err != cudaSuccess) return err;
      int cluster = 1;
      while (cluster < chunks && cluster < kClusterMost) cluster *= 2;
      return launch_cluster(kernel, cluster, kClusterThreads, 0, stream, list, partial, max_norm, out);
    }
  }
  for (int at = 0; at < n_tensors;) {
    const int chunks = fill(list, tensors, n_tensors, kBlockThreads, &at);
    if (chunks == 0) continue;
    const int resident = num_sms * 5;
    const int shares = most > resident && chunks / resident < kLongShare ? resident : most;
    const int grid = chunks < shares ? chunks : shares;
    if (blocks + grid > kGradNormMaxBlocks) return cudaErrorInvalidValue;
    squares_kernel<kCapacity, kBlockThreads>
        <<<grid, kBlockThreads, 0, stream>>>(list, partial + blocks, max_norm, nullptr);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    blocks += grid;
  }
  if (blocks == 0) {  // nothing to add up: the kernel has no other to wait for
    norm_kernel<<<1, kBlockThreads, 0, stream>>>(partial, blocks, max_norm, out);
    return cudaGetLastError();
  }
  return launch_dependent(norm_kernel, 1, kBlockThreads, 0, stream, partial, blocks, max_norm, out);
}

// Capacities of the kernels' lists: a call takes the smallest that holds its
// tensors (a launch copies the whole list), and as many launches of the
// largest as a longer list needs.
constexpr int kSmallList = 8, kMediumList = 48, kLargeList = kListMost;
static_assert(sizeof(List<kLargeList>) <= 32764, "kernel parameters");

}  // namespace

size_t grad_norm_workspace_bytes() { return align_up(kGradNormMaxBlocks * sizeof(double)); }

cudaError_t launch_grad_norm(const moe_adamw_tensor_t* tensors, int n_tensors, float max_norm, float* out,
                             double* partial, int num_sms, cudaStream_t stream) {
  if (n_tensors <= kSmallList) return norm_all<kSmallList>(tensors, n_tensors, max_norm, out, partial, num_sms, stream);
  if (n_tensors <= kMediumList) return norm_all<kMediumList>(tensors, n_tensors, max_norm, out, partial, num_sms, stream);
  return norm_all<kLargeList>(tensors, n_tensors, max_norm, out, partial, num_sms, stream);
}

cudaError_t launch_adamw(const moe_adamw_tensor_t* tensors, int n_tensors, const moe_adamw_hyper_t* hyper,
                         const moe_adamw_hyper_t* hyper_dev, const float* grad_scale, cudaStream_t stream) {
  if (n_tensors <= kSmallList) return adamw_all<kSmallList>(tensors, n_tensors, hyper, hyper_dev, grad_scale, stream);
  if (n_tensors <= kMediumList) return adamw_all<kMediumList>(tensors, n_tensors, hyper, hyper_dev, grad_scale, stream);
  return adamw_all<kLargeList>(tensors, n_tensors, hyper, hyper_dev, grad_scale, stream);
}

}  // namespace moe
