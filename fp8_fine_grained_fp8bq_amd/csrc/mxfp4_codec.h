// MXFP4 tile codec: the E8M0 scale byte of a tile from its largest magnitude
// and the E2M1 codes of values with that scale, shared by every kernel that
// writes MXFP4 operands.
//
// A tile's amax is the integer maximum of its magnitude bits (they order
// like the values; NaN and infinities come out on top). With E the exponent
// field of amax, floor(log2(amax)) - 2 + 127 is E - 2, cut off at 0 (subnormal
// amax included: E = 0).
// v_cvt_scalef32_pk_fp4_{f32,f16,bf16} divide two values by the power of two in
// an fp32 scale, round to nearest even, saturate to 6 and keep the sign, also
// with the subnormal scale 2^-127 (tests/test_gpu_mxfp4.py runs every midpoint
// and its neighbours under the smallest and largest scales of each type). The
// 16-bit forms spare the widening and the magnitudes are compared two at a
// time, so an element costs about two instructions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bq {

constexpr uint32_t kMxNan = 0xFFu;

template <bool NOSAT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  if (amax >= 0x7F800000u) return kMxNan;
  // NOSAT: one more where amax > 1.5 * 2^floor(log2 amax), i.e. > 6 * 2^e
  const int e = (int)(amax >> 23) - 2 + ((NOSAT && (amax & 0x7FFFFFu) > 0x400000u) ? 1 : 0);
  return e < 0 ? 0u : (uint32_t)e;
}
// 2^e of a scale byte (2^-127 is subnormal, 0xFF is NaN).
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return byte == kMxNan ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}
__device__ __forceinline__ uint32_t mx_mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Codes of eight consecutive values, the first in the low four bits: fp32, or
// pairs of bf16 / fp16 (the first in the low half of a dword).
__device__ __forceinline__ uint32_t mx_codes8(const float* v, uint32_t byte) {
  const float sc = mx_scale(byte);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], sc, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], sc, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], sc, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], sc, 3);
  return byte == kMxNan ? 0u : r;
}
typedef __bf16 mx_bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 mx_fp16x2 __attribute__((ext_vector_type(2)));
template <bool BF16>
__device__ __forceinline__ uint32_t mx_codes8(const uint32_t (&w)[4], uint32_t byte) {
  const float sc = mx_scale(byte);
  uint32_t r = 0;
  if constexpr (BF16) {
    mx_bf16x2 p[4];
    __builtin_memcpy(p, w, 16);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, p[0], sc, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, p[1], sc, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, p[2], sc, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, p[3], sc, 3);
  } else {
    mx_fp16x2 p[4];
    __builtin_memcpy(p, w, 16);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, p[0], sc, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, p[1], sc, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, p[2], sc, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, p[3], sc, 3);
  }
  return byte == kMxNan ? 0u : r;
}
// Larger magnitudes of two pairs of 16-bit floats, as pairs of magnitude bits.
typedef unsigned short mx_u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t mx_max_pairs(uint32_t mags, uint32_t w) {
  const uint32_t v = w & 0x7FFF7FFFu;
  mx_u16x2 a, b;
  __builtin_memcpy(&a, &mags, 4);
  __builtin_memcpy(&b, &v, 4);
  a = __builtin_elementwise_max(a, b);
  __builtin_memcpy(&mags, &a, 4);
  return mags;
}
// fp32 magnitude bits of 16-bit magnitude bits.
template <bool BF16>
__device__ __forceinline__ uint32_t mx_mag16(uint32_t m) {
  if constexpr (BF16) return m << 16;
  const uint16_t h = (uint16_t)m;
  _Float16 f;
  __builtin_memcpy(&f, &h, 2);
  return __float_as_uint((float)f) & 0x7FFFFFFFu;
}

}  // namespace fp8bq
