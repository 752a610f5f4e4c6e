// MXFP4 tile codec: the E8M0 scale byte of a tile from its largest magnitude
// and the E2M1 codes of values with that scale, shared by every kernel that
// writes MXFP4 operands.
//
// A tile's amax is the integer maximum of its fp32 magnitude bits (they order
// like the values; NaN and infinities come out on top). With E the exponent
// field of amax, floor(log2(amax)) - 2 + 127 is E - 2, cut off at 0 (subnormal
// amax included: E = 0). The quotient x * 2^-e is one product with the power
// of two whose exponent field is 254 - byte, a normal number for every byte
// that a finite amax gives (0 .. 253), so the product is exact unless it
// falls below 2^-126, far under the smallest midpoint (0.25).
// v_cvt_scalef32_pk_fp4_f32 with scale 1 rounds to nearest even, saturates to
// 6 and keeps the sign (tests/test_gpu_mxfp4.py runs every midpoint and its
// neighbours).
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
// What a value is multiplied by before it is rounded; 0 for a NaN tile (its
// codes are cleared by mx_codes8).
__device__ __forceinline__ float mx_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// 2^e of a scale byte (2^-127 is subnormal, 0xFF is NaN).
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return byte == kMxNan ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}
__device__ __forceinline__ uint32_t mx_mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Codes of eight consecutive values, the first in the low four bits.
__device__ __forceinline__ uint32_t mx_codes8(const float* v, uint32_t byte) {
  const float inv = mx_inverse(byte);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0] * inv, v[1] * inv, 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2] * inv, v[3] * inv, 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4] * inv, v[5] * inv, 1.0f, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6] * inv, v[7] * inv, 1.0f, 3);
  return byte == kMxNan ? 0u : r;
}

}  // namespace fp8bq
