// Argument checks that the files of entry points share (host only).
#pragma once

#include "../../include/fp8bq.h"

#include <hip/hip_runtime.h>

#include "entry.h"

namespace fp8bq {

constexpr int64_t kMaxSide = (int64_t)1 << 31;    // rows, columns: indices fit 32 bits
constexpr int64_t kMaxLd = (int64_t)1 << 23;      // bytes of a code row: 256 rows within 2 GiB
constexpr int64_t kMaxRouted = (int64_t)1 << 30;  // dispatched rows, choices

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int64_t chunks_of(int64_t k) { return (k - 1) / 256 + 1; }
inline int elem_bytes(int dtype) { return dtype == FP8BQ_FP32 ? 4 : 2; }
inline bool bad_dtype(int t) { return t != FP8BQ_BF16 && t != FP8BQ_FP16 && t != FP8BQ_FP32; }

inline int launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return entry_fail(FP8BQ_E_HIP, "%s: launch failed: %s", what, hipGetErrorString(e));
  return FP8BQ_OK;
}

// One code matrix [rows, k] with its scales.
inline int check_codes(const char* who, const char* name, const void* q, int64_t ldq, const void* s, int64_t lds,
                       int64_t rows, int64_t k) {
  if (!q || !s) return entry_fail(FP8BQ_E_INVAL, "%s: null codes or scales of %s", who, name);
  if (ldq < 128 * chunks_of(k))
    return entry_fail(FP8BQ_E_INVAL, "%s: ld of %s (%lld bytes) < 128 * ceil(k / 256)", who, name, (long long)ldq);
  if (lds < rows) return entry_fail(FP8BQ_E_INVAL, "%s: scale ld of %s must be >= its rows", who, name);
  if (ldq >= kMaxLd || lds >= kMaxSide / 8) return entry_fail(FP8BQ_E_SHAPE, "%s: ld of %s too large", who, name);
  if (!aligned(q, 16) || ldq % 16 || !aligned(s, 8))
    return entry_fail(FP8BQ_E_ALIGN, "%s: codes of %s must be 16-byte aligned with ld a multiple of 16, scales 8-byte "
                      "aligned", who, name);
  return FP8BQ_OK;
}

}  // namespace fp8bq
