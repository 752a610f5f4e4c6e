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

// 16 bytes at a time whatever the alignment: global accesses need no more than
// the element's on gfx950 (a wave's unaligned one touches one more line).
typedef uint32_t u32x4_unaligned __attribute__((ext_vector_type(4), aligned(1)));
template <class V>
__device__ __forceinline__ V load_any(const void* p) {
  V v;
  __builtin_memcpy(&v, p, sizeof(V));
  return v;
}
// Results that are written whole, as they go by: marked as not worth keeping in
// the caches. Us without and with, called back to back: codes of 8192 tokens of 7168
// columns dispatched to 64 experts 116 / 105; rows of 16384 x 7168 normalised, with
// a residual and codes 193 / 189, the gradient 189 / 184; of 4096 x 7168 49 / 43 (53 /
// 51 where no operand is in a cache), but with codes alone 36 / 38.6 (45 / 44). Loads
// so marked were slower by a fifth to a third wherever an operand still was in a
// cache, and faster only far beyond their size.
template <class V>
__device__ __forceinline__ void stream_store(void* p, const V& v) {
  if constexpr (sizeof(V) % 16 == 0) {
    u32x4_unaligned t[sizeof(V) / 16];
    __builtin_memcpy(t, &v, sizeof(V));
#pragma unroll
    for (int i = 0; i < (int)(sizeof(V) / 16); ++i) __builtin_nontemporal_store(t[i], static_cast<u32x4_unaligned*>(p) + i);
  } else {
    __builtin_memcpy(p, &v, sizeof(V));
  }
}

// Neighbouring elements, and eight of them as fp32 and back.
template <int T, int N> struct Some { typename Elem<T>::type e[N]; };
template <int T> struct Raw8 { uint32_t w[2 * Elem<T>::kBytes]; };
template <int T>
__device__ __forceinline__ Raw8<T> load8(const typename Elem<T>::type* p) {
  return load_any<Raw8<T>>(p);
}
template <int T>
__device__ __forceinline__ void values8(const Raw8<T>& r, float (&v)[8]) {
  typename Elem<T>::type e[8];
  __builtin_memcpy(e, &r, sizeof(r));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = Elem<T>::value(e[i]);
}
template <int T>
__device__ __forceinline__ Raw8<T> round8(const float (&v)[8]) {
  typename Elem<T>::type e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = Elem<T>::round(v[i]);
  Raw8<T> r;
  __builtin_memcpy(&r, e, sizeof(r));
  return r;
}

}  // namespace fp8bq
