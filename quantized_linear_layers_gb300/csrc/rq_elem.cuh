// rq_elem.cuh -- elements of f32, f16 and bf16 rows as floats, and back.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace rq {

__device__ __forceinline__ float elem_float(float x) { return x; }
__device__ __forceinline__ float elem_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float elem_float(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T float_elem(float x);
template <>
__device__ __forceinline__ float float_elem<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __half float_elem<__half>(float x) {
  return __float2half_rn(x);
}
template <>
__device__ __forceinline__ __nv_bfloat16 float_elem<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// Two 16-bit elements of a word (the first in its low half) as floats, and back.
template <typename T>
__device__ __forceinline__ float2 word_floats(uint32_t w);
template <>
__device__ __forceinline__ float2 word_floats<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 word_floats<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t floats_word(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t floats_word<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t floats_word<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// V consecutive elements: one element, or whole 16-byte groups.
template <typename T, int V>
__device__ __forceinline__ void load_elems(const T* p, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = elem_float(*p);
  } else {
    constexpr int kPer = 16 / (int)sizeof(T);
    static_assert(V % kPer == 0, "whole 16-byte groups");
#pragma unroll
    for (int i = 0; i < V; i += kPer) {
      const uint4 u = *reinterpret_cast<const uint4*>(p + i);
      const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[i + j] = elem_float(t[j]);
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_elems(T* p, const float (&x)[V]) {
  if constexpr (V == 1) {
    *p = float_elem<T>(x[0]);
  } else {
    constexpr int kPer = 16 / (int)sizeof(T);
    static_assert(V % kPer == 0, "whole 16-byte groups");
#pragma unroll
    for (int i = 0; i < V; i += kPer) {
      alignas(16) T t[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) t[j] = float_elem<T>(x[i + j]);
      *reinterpret_cast<uint4*>(p + i) = *reinterpret_cast<const uint4*>(t);
    }
  }
}

}  // namespace rq
