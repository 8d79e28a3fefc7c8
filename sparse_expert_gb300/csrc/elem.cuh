// Element types of the training-step kernels (layer norm, optimizer): fp32,
// bf16 and fp16 values read from memory, computed on in fp32, rounded to
// nearest even when stored.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace moe {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// One 32-bit word holds one fp32 value or two 16-bit ones.
template <typename T>
struct Word;
template <>
struct Word<float> {
  static constexpr int kValues = 1;
  __device__ static __forceinline__ void unpack(uint32_t u, float* v) { v[0] = __uint_as_float(u); }
  __device__ static __forceinline__ uint32_t pack(const float* v) { return __float_as_uint(v[0]); }
};
template <>
struct Word<__nv_bfloat16> {
  static constexpr int kValues = 2;
  __device__ static __forceinline__ void unpack(uint32_t u, float* v) {
    v[0] = __uint_as_float(u << 16);
    v[1] = __uint_as_float(u & 0xffff0000u);
  }
  __device__ static __forceinline__ uint32_t pack(const float* v) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[0], v[1]);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
};
template <>
struct Word<__half> {
  static constexpr int kValues = 2;
  __device__ static __forceinline__ void unpack(uint32_t u, float* v) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
    v[0] = f.x;
    v[1] = f.y;
  }
  __device__ static __forceinline__ uint32_t pack(const float* v) {
    const __half2 p = __floats2half2_rn(v[0], v[1]);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
};

// The 16 bytes of a chunk as fp32 values, and back.
template <typename T>
constexpr int kChunk = 16 / static_cast<int>(sizeof(T));

template <typename T>
__device__ __forceinline__ void unpack_chunk(const uint4& u, float* v) {
  constexpr int k = Word<T>::kValues;
  Word<T>::unpack(u.x, v);
  Word<T>::unpack(u.y, v + k);
  Word<T>::unpack(u.z, v + 2 * k);
  Word<T>::unpack(u.w, v + 3 * k);
}

template <typename T>
__device__ __forceinline__ uint4 pack_chunk(const float* v) {
  constexpr int k = Word<T>::kValues;
  return make_uint4(Word<T>::pack(v), Word<T>::pack(v + k), Word<T>::pack(v + 2 * k), Word<T>::pack(v + 3 * k));
}

// Two fp32 operations in one instruction, each rounded on its own.
__device__ __forceinline__ uint64_t pair_bits(float2 v) {
  return static_cast<uint64_t>(__float_as_uint(v.x)) | static_cast<uint64_t>(__float_as_uint(v.y)) << 32;
}
__device__ __forceinline__ float2 bits_pair(uint64_t u) {
  return make_float2(__uint_as_float(static_cast<uint32_t>(u)), __uint_as_float(static_cast<uint32_t>(u >> 32)));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return bits_pair(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return bits_pair(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair_bits(a)), "l"(pair_bits(b)), "l"(pair_bits(c)));
  return bits_pair(r);
}

// A chunk as pairs, and back.
template <typename T>
constexpr int kPairs = kChunk<T> / 2;

template <typename T>
__device__ __forceinline__ void unpack_pairs(const uint4& u, float2* v) {
  float f[kChunk<T>];
  unpack_chunk<T>(u, f);
#pragma unroll
  for (int i = 0; i < kPairs<T>; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
}

template <typename T>
__device__ __forceinline__ uint4 pack_pairs(const float2* v) {
  float f[kChunk<T>];
#pragma unroll
  for (int i = 0; i < kPairs<T>; ++i) f[2 * i] = v[i].x, f[2 * i + 1] = v[i].y;
  return pack_chunk<T>(f);
}

// The chunk's sums, each rounded to the type: for the 16-bit types the fp32
// sum of two of their values rounds to the same value (24 >= 2 * 11 + 2).
template <typename T>
__device__ __forceinline__ uint32_t add_word(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t add_word<float>(uint32_t a, uint32_t b) {
  return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
}
template <>
__device__ __forceinline__ uint32_t add_word<__nv_bfloat16>(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t add_word<__half>(uint32_t a, uint32_t b) {
  const __half2 r = __hadd2_rn(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint4 add_chunks(const uint4& a, const uint4& b) {
  return make_uint4(add_word<T>(a.x, b.x), add_word<T>(a.y, b.y), add_word<T>(a.z, b.z), add_word<T>(a.w, b.w));
}

// Sum over the warp, the same value on every lane.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

}  // namespace moe
