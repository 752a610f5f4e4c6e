// Elements of the three types that the MXFP4, routing and norm operators take
// (fp8bq_dtype): their storage, their value in fp32, and fp32 rounded to them
// (to nearest, ties to even).
#pragma once

#include "../../include/fp8bq.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bq {

template <int T> struct Elem;
template <> struct Elem<FP8BQ_BF16> {
  using type = uint16_t;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
  static __device__ __forceinline__ uint16_t round(float v) {
    const __bf16 b = (__bf16)v;
    uint16_t r;
    __builtin_memcpy(&r, &b, 2);
    return r;
  }
};
template <> struct Elem<FP8BQ_FP16> {
  using type = uint16_t;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float value(uint16_t b) {
    _Float16 h;
    __builtin_memcpy(&h, &b, 2);
    return (float)h;
  }
  static __device__ __forceinline__ uint16_t round(float v) {
    const _Float16 h = (_Float16)v;
    uint16_t r;
    __builtin_memcpy(&r, &h, 2);
    return r;
  }
};
template <> struct Elem<FP8BQ_FP32> {
  using type = float;
  static constexpr int kBytes = 4;
  static __device__ __forceinline__ float value(float b) { return b; }
  static __device__ __forceinline__ float round(float v) { return v; }
};

// Eight neighbouring elements as fp32, and back. The memory may be aligned to
// the element only: global loads and stores of 16 bytes need no more on gfx950
// (a wave's unaligned access touches one more line at each end).
template <int T> struct Raw8 { uint32_t w[2 * Elem<T>::kBytes]; };
template <int T>
__device__ __forceinline__ Raw8<T> load8(const typename Elem<T>::type* p) {
  Raw8<T> r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}
template <int T>
__device__ __forceinline__ void values8(const Raw8<T>& r, float (&v)[8]) {
  typename Elem<T>::type e[8];
  __builtin_memcpy(e, &r, sizeof(r));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = Elem<T>::value(e[i]);
}
template <int T>
__device__ __forceinline__ void store8(typename Elem<T>::type* p, const float (&v)[8]) {
  typename Elem<T>::type e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = Elem<T>::round(v[i]);
  __builtin_memcpy(p, e, sizeof(e));
}

}  // namespace fp8bq
