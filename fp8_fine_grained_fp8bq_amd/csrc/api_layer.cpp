// C-ABI entry points of the operators around a layer's Linears: argument
// validation (host only, before any HIP call), the device check, and dispatch
// to the kernel launchers. The operations are specified in include/fp8bq.h.
#include "../../include/fp8bq.h"

#include <hip/hip_runtime.h>
#include <math.h>

#include "entry_checks.h"
#include "layer.h"

namespace {

using namespace fp8bq;

bool bad_ld(int64_t ld, int64_t rows) { return ld > INT64_MAX / 4 / rows; }

int check_norm(const char* who, int type, int wtype, int64_t rows, int64_t cols) {
  if (bad_dtype(type) || bad_dtype(wtype))
    return entry_fail(FP8BQ_E_INVAL, "%s: types must be BF16, FP16 or FP32, got %d and %d", who, type, wtype);
  if (rows <= 0 || cols <= 0) return entry_fail(FP8BQ_E_INVAL, "%s: rows and cols must be positive", who);
  if (rows >= kMaxSide || cols > kNormMaxCols)
    return entry_fail(FP8BQ_E_SHAPE, "%s: too large (rows below 2^31, cols up to %d)", who, kNormMaxCols);
  return FP8BQ_OK;
}

// A matrix of rows: its pointer is not null.
int check_rows(const char* who, const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int bytes) {
  if (!p) return entry_fail(FP8BQ_E_INVAL, "%s: null %s", who, name);
  if (ld < cols) return entry_fail(FP8BQ_E_INVAL, "%s: ld of %s (%lld) < cols (%lld)", who, name, (long long)ld, (long long)cols);
  if (bad_ld(ld, rows)) return entry_fail(FP8BQ_E_SHAPE, "%s: ld of %s too large", who, name);
  if (!aligned(p, bytes)) return entry_fail(FP8BQ_E_ALIGN, "%s: %s must be aligned to its element", who, name);
  return FP8BQ_OK;
}

// What the three routing operators share. `none`: there may be no rows.
int check_plan(const char* who, int64_t tokens, int64_t rows, int64_t cols, int64_t topk, const int32_t* pos, bool none = false) {
  if (tokens <= 0 || rows < 0 || (rows == 0 && !none) || cols <= 0 || topk <= 0) return entry_fail(FP8BQ_E_INVAL, "%s: sizes must be positive", who);
  if (!pos) return entry_fail(FP8BQ_E_INVAL, "%s: null pos", who);
  if (!aligned(pos, 4)) return entry_fail(FP8BQ_E_ALIGN, "%s: pos must be 4-byte aligned", who);
  if (tokens >= kMaxRouted || topk >= kMaxRouted || tokens * topk >= kMaxRouted || rows >= kMaxRouted || cols >= kMaxSide)
    return entry_fail(FP8BQ_E_SHAPE, "%s: too large", who);
  return FP8BQ_OK;
}

int check_gate(const char* who, const float* w, int64_t tokens, int64_t topk, int64_t ldw) {
  if (ldw < topk) return entry_fail(FP8BQ_E_INVAL, "%s: ldw < topk", who);
  if (bad_ld(ldw, tokens)) return entry_fail(FP8BQ_E_SHAPE, "%s: ldw too large", who);
  if (!aligned(w, 4)) return entry_fail(FP8BQ_E_ALIGN, "%s: weight must be 4-byte aligned", who);
  return FP8BQ_OK;
}

int gemv(const char* who, bool grouped, int32_t groups, const int32_t* row_off, int64_t m, int64_t n, int64_t k, const void* x,
         int xtype, int64_t xrows, int64_t ldx, const int32_t* src, const void* b, int64_t ldb, const void* sb, int64_t ldsb,
         void* out, int otype, int64_t ldo, void* stream) {
  if (m <= 0 || n <= 0 || k <= 0 || xrows <= 0) return entry_fail(FP8BQ_E_INVAL, "%s: sizes must be positive", who);
  if (bad_dtype(xtype) || bad_dtype(otype))
    return entry_fail(FP8BQ_E_INVAL, "%s: types must be BF16, FP16 or FP32, got %d and %d", who, xtype, otype);
  if (grouped) {
    if (!row_off) return entry_fail(FP8BQ_E_INVAL, "%s: null row_off", who);
    if (groups < 1 || groups > 256) return entry_fail(FP8BQ_E_SHAPE, "%s: groups must be 1 .. 256, got %d", who, groups);
    if (!src && xrows < m) return entry_fail(FP8BQ_E_INVAL, "%s: xrows < rows without src", who);
    if (!aligned(row_off, 4) || !aligned(src, 4))
      return entry_fail(FP8BQ_E_ALIGN, "%s: row_off and src must be 4-byte aligned", who);
  }
  // workgroups of up to 256 threads for 16 rows of the weight and up to 16 of x; 65535 row tiles (of two rows where m is 2 at most)
  if (m > 65535 * (int64_t)16 || xrows >= kMaxSide || n >= ((int64_t)1 << 26) || k >= ((int64_t)1 << 28) ||
      (n / 16 + 1) * (grouped ? groups : m / 16 + 1) >= ((int64_t)1 << 22))
    return entry_fail(FP8BQ_E_SHAPE, "%s: too large", who);
  if (int e = check_rows(who, "x", x, xrows, k, ldx, elem_bytes(xtype))) return e;
  if (int e = check_codes(who, "b", b, ldb, sb, ldsb, n, k)) return e;
  if (int e = check_rows(who, "out", out, m, n, ldo, elem_bytes(otype))) return e;
  if (int e = entry_device()) return e;
  const GemvArgs p{m, n, k, x, xrows, ldx, static_cast<const uint8_t*>(b), ldb, static_cast<const uint8_t*>(sb), ldsb,
                   out, otype, ldo, grouped ? groups : 0, row_off, src};
  return launched(launch_gemv_mxfp4(p, xtype, reinterpret_cast<hipStream_t>(stream)), who);
}

}  // namespace

extern "C" {

int fp8bq_rmsnorm(const void* x, int xtype, int64_t rows, int64_t cols, int64_t ldx, const void* residual, int64_t ldr,
                  const void* weight, int wtype, float eps, void* h, int64_t ldh, void* y, int64_t ldy, void* q,
                  int64_t ldq, float* s, int64_t lds, float* rstd, int flags, void* stream) {
  const char* who = "rmsnorm";
  if (int e = check_norm(who, xtype, wtype, rows, cols)) return e;
  if (flags & ~FP8BQ_SCALE_POW2) return entry_fail(FP8BQ_E_INVAL, "%s: unknown flags %d", who, flags);
  if (!(eps >= 0.f) || isinf(eps)) return entry_fail(FP8BQ_E_INVAL, "%s: eps must be finite and not negative", who);
  if (!weight) return entry_fail(FP8BQ_E_INVAL, "%s: null weight", who);
  if (!residual != !h) return entry_fail(FP8BQ_E_INVAL, "%s: residual and h go together", who);
  if (!q != !s) return entry_fail(FP8BQ_E_INVAL, "%s: q and s go together", who);
  if (!y && !q) return entry_fail(FP8BQ_E_INVAL, "%s: no output asked for", who);
  const int bytes = elem_bytes(xtype);
  if (int e = check_rows(who, "x", x, rows, cols, ldx, bytes)) return e;
  if (residual) {
    if (int e = check_rows(who, "residual", residual, rows, cols, ldr, bytes)) return e;
    if (int e = check_rows(who, "h", h, rows, cols, ldh, bytes)) return e;
  }
  if (y)
    if (int e = check_rows(who, "y", y, rows, cols, ldy, bytes)) return e;
  if (q) {
    if (cols % 128) return entry_fail(FP8BQ_E_SHAPE, "%s: cols (%lld) must be a multiple of 128", who, (long long)cols);
    if (int e = check_rows(who, "q", q, rows, cols, ldq, 16)) return e;
    if (ldq % 16) return entry_fail(FP8BQ_E_ALIGN, "%s: ldq must be a multiple of 16", who);
    if (int e = check_rows(who, "s", s, cols / 128, rows, lds, 4)) return e;
  }
  if (!aligned(weight, elem_bytes(wtype)) || !aligned(rstd, 4))
    return entry_fail(FP8BQ_E_ALIGN, "%s: weight must be aligned to its element, rstd to 4 bytes", who);
  if (int e = entry_device()) return e;
  const NormArgs a{x, rows, (int)cols, ldx, residual, ldr, weight, wtype, eps, h, ldh, y, ldy,
                   static_cast<uint8_t*>(q), ldq, s, lds, rstd};
  return launched(launch_rmsnorm(a, xtype, (flags & FP8BQ_SCALE_POW2) != 0, reinterpret_cast<hipStream_t>(stream)), who);
}

int fp8bq_rmsnorm_grad_workspace_size(int64_t rows, int64_t cols, int64_t* bytes) {
  const char* who = "rmsnorm_grad_workspace_size";
  if (!bytes) return entry_fail(FP8BQ_E_INVAL, "%s: null bytes", who);
  if (int e = check_norm(who, FP8BQ_BF16, FP8BQ_BF16, rows, cols)) return e;
  *bytes = norm_grad_parts(rows, cols) * cols * 4;
  return FP8BQ_OK;
}

int fp8bq_rmsnorm_grad(const void* dy, int type, int64_t rows, int64_t cols, int64_t lddy, const void* h, int64_t ldh,
                       const void* weight, int wtype, const float* rstd, const void* dh, int64_t lddh, void* dx,
                       int64_t lddx, float* dweight, void* workspace, void* stream) {
  const char* who = "rmsnorm_grad";
  if (int e = check_norm(who, type, wtype, rows, cols)) return e;
  if (!weight || !rstd || !dweight || !workspace) return entry_fail(FP8BQ_E_INVAL, "%s: null pointer", who);
  const int bytes = elem_bytes(type);
  if (int e = check_rows(who, "dy", dy, rows, cols, lddy, bytes)) return e;
  if (int e = check_rows(who, "h", h, rows, cols, ldh, bytes)) return e;
  if (dh)
    if (int e = check_rows(who, "dh", dh, rows, cols, lddh, bytes)) return e;
  if (int e = check_rows(who, "dx", dx, rows, cols, lddx, bytes)) return e;
  if (!aligned(weight, elem_bytes(wtype)) || !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(workspace, 4))
    return entry_fail(FP8BQ_E_ALIGN, "%s: misaligned pointer", who);
  if (int e = entry_device()) return e;
  const NormGradArgs a{dy, rows, (int)cols, lddy, h, ldh, weight, wtype, rstd, dh, lddh, dx, lddx, dweight,
                       static_cast<float*>(workspace)};
  return launched(launch_rmsnorm_grad(a, type, reinterpret_cast<hipStream_t>(stream)), who);
}

int fp8bq_moe_dispatch(const void* x, int elem, int64_t tokens, int64_t cols, int64_t ldx, const float* s, int64_t lds,
                       const int32_t* pos, int64_t topk, const int32_t* src, int64_t rows, void* out, int64_t ldo,
                       float* so, int64_t ldso, void* stream) {
  const char* who = "moe_dispatch";
  if (elem != 1 && elem != 2 && elem != 4) return entry_fail(FP8BQ_E_INVAL, "%s: elem must be 1, 2 or 4, got %d", who, elem);
  if (int e = check_plan(who, tokens, rows, cols, topk, pos)) return e;
  if (!src) return entry_fail(FP8BQ_E_INVAL, "%s: null src", who);
  if (!s != !so) return entry_fail(FP8BQ_E_INVAL, "%s: s and so go together", who);
  if (int e = check_rows(who, "x", x, tokens, cols, ldx, elem)) return e;
  if (int e = check_rows(who, "out", out, rows, cols, ldo, elem)) return e;
  if (s) {
    if (elem != 1) return entry_fail(FP8BQ_E_INVAL, "%s: scales go with 8-bit codes", who);
    if (cols % 128) return entry_fail(FP8BQ_E_SHAPE, "%s: cols (%lld) must be a multiple of 128", who, (long long)cols);
    if (int e = check_rows(who, "s", s, cols / 128, tokens, lds, 4)) return e;
    if (int e = check_rows(who, "so", so, cols / 128, rows, ldso, 4)) return e;
  }
  if (!aligned(src, 4)) return entry_fail(FP8BQ_E_ALIGN, "%s: src must be 4-byte aligned", who);
  if (int e = entry_device()) return e;
  const MoeDispatchArgs a{static_cast<const uint8_t*>(x), elem, tokens, cols, ldx, s, lds, pos, (int)topk, src, rows,
                          static_cast<uint8_t*>(out), ldo, so, ldso};
  return launched(launch_moe_dispatch(a, reinterpret_cast<hipStream_t>(stream)), who);
}

int fp8bq_moe_combine(const void* y, int type, int64_t rows, int64_t cols, int64_t ldy, const int32_t* pos, int64_t tokens,
                      int64_t topk, const float* weight, int64_t ldw, const void* base, int64_t ldb, void* out, int64_t ldo,
                      void* stream) {
  const char* who = "moe_combine";
  if (bad_dtype(type)) return entry_fail(FP8BQ_E_INVAL, "%s: type must be BF16, FP16 or FP32, got %d", who, type);
  if (int e = check_plan(who, tokens, rows, cols, topk, pos, !y)) return e;
  if (rows)
    if (int e = check_rows(who, "y", y, rows, cols, ldy, elem_bytes(type))) return e;
  if (weight)
    if (int e = check_gate(who, weight, tokens, topk, ldw)) return e;
  if (base)
    if (int e = check_rows(who, "base", base, tokens, cols, ldb, elem_bytes(type))) return e;
  if (int e = check_rows(who, "out", out, tokens, cols, ldo, elem_bytes(type))) return e;
  if (int e = entry_device()) return e;
  const MoeCombineArgs a{y, rows, cols, ldy, pos, tokens, (int)topk, weight, ldw, base, ldb, out, ldo};
  return launched(launch_moe_combine(a, type, reinterpret_cast<hipStream_t>(stream)), who);
}

int fp8bq_moe_combine_grad(const void* dout, int type, int64_t tokens, int64_t cols, int64_t lddout, const void* y,
                           int64_t rows, int64_t ldy, const int32_t* pos, int64_t topk, const float* weight, int64_t ldw,
                           const int32_t* src, void* dy, int64_t lddy, float* dweight, void* stream) {
  const char* who = "moe_combine_grad";
  if (bad_dtype(type)) return entry_fail(FP8BQ_E_INVAL, "%s: type must be BF16, FP16 or FP32, got %d", who, type);
  if (int e = check_plan(who, tokens, rows, cols, topk, pos, !y)) return e;
  if (!weight || (rows && !src) || !dweight) return entry_fail(FP8BQ_E_INVAL, "%s: null pointer", who);
  if (int e = check_gate(who, weight, tokens, topk, ldw)) return e;
  if (int e = check_rows(who, "dout", dout, tokens, cols, lddout, elem_bytes(type))) return e;
  if (rows) {
    if (int e = check_rows(who, "y", y, rows, cols, ldy, elem_bytes(type))) return e;
    if (int e = check_rows(who, "dy", dy, rows, cols, lddy, elem_bytes(type))) return e;
  }
  if (!aligned(src, 4) || !aligned(dweight, 4)) return entry_fail(FP8BQ_E_ALIGN, "%s: src and dweight must be 4-byte aligned", who);
  if (int e = entry_device()) return e;
  const MoeCombineGradArgs a{dout, tokens, cols, lddout, y, rows, ldy, pos, (int)topk, weight, ldw, src, dy, lddy, dweight};
  return launched(launch_moe_combine_grad(a, type, reinterpret_cast<hipStream_t>(stream)), who);
}

int fp8bq_gemv_mxfp4(int64_t m, int64_t n, int64_t k, const void* x, int xtype, int64_t ldx, const void* b, int64_t ldb,
                     const void* sb, int64_t ldsb, void* out, int otype, int64_t ldo, void* stream) {
  return gemv("gemv_mxfp4", false, 0, nullptr, m, n, k, x, xtype, m, ldx, nullptr, b, ldb, sb, ldsb, out, otype, ldo, stream);
}

int fp8bq_grouped_gemv_mxfp4(int32_t groups, const int32_t* row_off, int64_t rows, int64_t n, int64_t k, const void* x,
                             int xtype, int64_t xrows, int64_t ldx, const int32_t* src, const void* b, int64_t ldb,
                             const void* sb, int64_t ldsb, void* out, int otype, int64_t ldo, void* stream) {
  return gemv("grouped_gemv_mxfp4", true, groups, row_off, rows, n, k, x, xtype, xrows, ldx, src, b, ldb, sb, ldsb, out,
              otype, ldo, stream);
}

}  // extern "C"
