// C-ABI entry points of the MXFP4 operators and the routing of tokens to
// experts: argument validation (host only, before any HIP call), the device
// check, and dispatch to the kernel launchers. The operations and their
// layouts are specified in include/fp8bq.h.
#include "../../include/fp8bq.h"

#include <hip/hip_runtime.h>

#include "entry_checks.h"
#include "mxfp4.h"

static_assert(FP8BQ_DISPATCH_WORKSPACE_ROW_BYTES == 4 * (fp8bq::kMxDispatchSlots + 1), "workspace size in the header");
static_assert(FP8BQ_MOE_PLAN_WORKSPACE_BYTES == fp8bq::kMoePlanMaxBlocks * 256 * 4, "workspace size in the header");

namespace {

using namespace fp8bq;

// Grids have fewer than 2^32 threads, that is 2^24 blocks of 256. Row form and
// read-back: at most one block for 16 rows of a chunk.
bool too_large(int64_t rows, int64_t cols) {
  return rows >= kMaxSide || chunks_of(cols) > 16383 || ((rows - 1) / 16 + 1) * chunks_of(cols) >= ((int64_t)1 << 24);
}
// Column form: whole 256 x 256 squares in blocks of 128 rows of 128 bytes
// (rows and cols as too_large leaves them).
bool too_large_by_columns(int64_t rows, int64_t cols, int xtype) {
  return ((rows - 1) / 256 + 1) * chunks_of(cols) * (4 * elem_bytes(xtype)) >= ((int64_t)1 << 24);
}

int quant(const char* who, const void* x, int xtype, int64_t xrows, int64_t cols, int64_t ldx, const int32_t* src,
          bool indexed, int64_t rows, void* q, int64_t ldq, void* s, int64_t lds, void* qt, int64_t ldqt, void* st,
          int64_t ldst, int flags, void* ws, void* stream) {
  if (!x || (indexed && !src)) return entry_fail(FP8BQ_E_INVAL, "%s: null pointer", who);
  if (bad_dtype(xtype)) return entry_fail(FP8BQ_E_INVAL, "%s: type must be BF16, FP16 or FP32, got %d", who, xtype);
  if (flags & ~FP8BQ_MX_NOSAT) return entry_fail(FP8BQ_E_INVAL, "%s: unknown flags %d", who, flags);
  if (rows <= 0 || cols <= 0 || xrows <= 0) return entry_fail(FP8BQ_E_INVAL, "%s: rows and cols must be positive", who);
  if (ldx < cols) return entry_fail(FP8BQ_E_INVAL, "%s: ldx (%lld) < cols (%lld)", who, (long long)ldx, (long long)cols);
  if (!q && !s && !qt && !st) return entry_fail(FP8BQ_E_INVAL, "%s: no output asked for", who);
  if (too_large(rows, cols) || xrows >= kMaxSide) return entry_fail(FP8BQ_E_SHAPE, "%s: too large", who);
  if (ldx > INT64_MAX / 4 / xrows) return entry_fail(FP8BQ_E_SHAPE, "%s: ldx too large", who);
  if (q || s)
    if (int e = check_codes(who, "the row form", q, ldq, s, lds, rows, cols)) return e;
  if (qt || st)
    if (int e = check_codes(who, "the transposed form", qt, ldqt, st, ldst, cols, rows)) return e;
  if (too_large(xrows, cols) || ((qt || st) && too_large_by_columns(rows, cols, xtype)))
    return entry_fail(FP8BQ_E_SHAPE, "%s: too large", who);
  if (!aligned(x, elem_bytes(xtype)) || !aligned(src, 4) || !aligned(ws, 16))
    return entry_fail(FP8BQ_E_ALIGN, "%s: x must be aligned to its element, src to 4 bytes, workspace to 16", who);
  if (int e = fp8bq::entry_device()) return e;
  const fp8bq::MxQuantArgs a{x, xrows, rows, cols, ldx, src,
                             static_cast<uint8_t*>(q), ldq, static_cast<uint8_t*>(s), lds,
                             static_cast<uint8_t*>(qt), ldqt, static_cast<uint8_t*>(st), ldst};
  // Reading each row once pays for two small launches and the slots.
  const bool once = ws && !qt && rows >= 2 * xrows;
  return launched(fp8bq::launch_quant_mxfp4(a, xtype, (flags & FP8BQ_MX_NOSAT) != 0,
                                            once ? static_cast<int32_t*>(ws) : nullptr,
                                            reinterpret_cast<hipStream_t>(stream)), who);
}

int gemm(const char* who, fp8bq::MxMode mode, int32_t groups, const int32_t* row_off, int64_t m, int64_t n, int64_t k,
         const void* a, int64_t lda, const void* sa, int64_t ldsa, const void* b, int64_t ldb, const void* sb,
         int64_t ldsb, void* out, int otype, int64_t ldo, void* stream) {
  if (m <= 0 || n <= 0 || k <= 0) return entry_fail(FP8BQ_E_INVAL, "%s: sizes must be positive", who);
  if (!out) return entry_fail(FP8BQ_E_INVAL, "%s: null output", who);
  if (otype != FP8BQ_BF16 && otype != FP8BQ_FP32)
    return entry_fail(FP8BQ_E_INVAL, "%s: output type must be BF16 or FP32, got %d", who, otype);
  if (ldo < n) return entry_fail(FP8BQ_E_INVAL, "%s: ldo must be >= n", who);
  if (mode != fp8bq::MX_DENSE) {
    if (!row_off) return entry_fail(FP8BQ_E_INVAL, "%s: null row_off", who);
    if (groups < 1 || groups > 256) return entry_fail(FP8BQ_E_SHAPE, "%s: groups must be 1 .. 256, got %d", who, groups);
    if (!aligned(row_off, 4)) return entry_fail(FP8BQ_E_ALIGN, "%s: row_off must be 4-byte aligned", who);
  }
  // tile counts (32 x 32 at the smallest) fit 31 bits
  if (m >= ((int64_t)1 << 28) || n >= ((int64_t)1 << 28) || k >= ((int64_t)1 << 28) || ldo >= ((int64_t)1 << 28) ||
      m / 32 + 257 > (((int64_t)1 << 31) - 1) / (n / 32 + 1) / (mode == fp8bq::MX_K ? groups : 1))
    return entry_fail(FP8BQ_E_SHAPE, "%s: too large", who);
  if (int e = check_codes(who, "a", a, lda, sa, ldsa, m, k)) return e;
  if (int e = check_codes(who, "b", b, ldb, sb, ldsb, n, k)) return e;
  if (!aligned(out, elem_bytes(otype)))
    return entry_fail(FP8BQ_E_ALIGN, "%s: out must be aligned to its element", who);
  if (int e = fp8bq::entry_device()) return e;
  const fp8bq::MxGemmArgs p{m, n, (int)chunks_of(k),
                            static_cast<const uint8_t*>(a), lda, static_cast<const uint8_t*>(sa), ldsa,
                            static_cast<const uint8_t*>(b), ldb, static_cast<const uint8_t*>(sb), ldsb,
                            out, ldo, groups, row_off};
  return launched(fp8bq::launch_gemm_mxfp4(p, mode, otype == FP8BQ_FP32, reinterpret_cast<hipStream_t>(stream)), who);
}

int check_balance(const char* who, const void* logits, int ltype, int64_t tokens, int64_t experts, int64_t ldl,
                  const int32_t* idx, int64_t topk, int64_t ldidx, const int32_t* seq_off, int64_t sequences, int score) {
  if (!logits || !idx) return entry_fail(FP8BQ_E_INVAL, "%s: null pointer", who);
  if (bad_dtype(ltype)) return entry_fail(FP8BQ_E_INVAL, "%s: type must be BF16, FP16 or FP32, got %d", who, ltype);
  if (score != FP8BQ_SOFTMAX && score != FP8BQ_SIGMOID)
    return entry_fail(FP8BQ_E_INVAL, "%s: score must be SOFTMAX or SIGMOID, got %d", who, score);
  if (tokens <= 0 || experts <= 0 || topk <= 0 || sequences <= 0)
    return entry_fail(FP8BQ_E_INVAL, "%s: sizes must be positive", who);
  if (!seq_off && sequences != 1) return entry_fail(FP8BQ_E_INVAL, "%s: null seq_off with %lld sequences", who, (long long)sequences);
  if (ldl < experts || ldidx < topk) return entry_fail(FP8BQ_E_INVAL, "%s: ld too small", who);
  if (experts > 1024 || sequences > 65534 || tokens >= kMaxSide || topk >= kMaxSide || tokens * topk >= kMaxSide ||
      ldl > INT64_MAX / 4 / tokens || ldidx > INT64_MAX / 4 / tokens)
    return entry_fail(FP8BQ_E_SHAPE, "%s: too large", who);
  if (!aligned(logits, elem_bytes(ltype)) || !aligned(idx, 4) || !aligned(seq_off, 4))
    return entry_fail(FP8BQ_E_ALIGN, "%s: misaligned pointer", who);
  return FP8BQ_OK;
}

fp8bq::MoeBalanceArgs balance_args(const void* logits, int64_t tokens, int64_t experts, int64_t ldl, const int32_t* idx,
                                   int64_t topk, int64_t ldidx, const int32_t* seq_off, int64_t sequences, float coef) {
  return {logits, ldl, tokens, (int)experts, (int)topk, idx, ldidx, seq_off, (int)sequences, coef};
}

}  // namespace

extern "C" {

int fp8bq_quant_mxfp4_1x32(const void* x, int xtype, int64_t rows, int64_t cols, int64_t ldx, void* q, int64_t ldq,
                           void* s, int64_t lds, void* qt, int64_t ldqt, void* st, int64_t ldst, int flags,
                           void* stream) {
  return quant("quant_mxfp4", x, xtype, rows, cols, ldx, nullptr, false, rows, q, ldq, s, lds, qt, ldqt, st, ldst,
               flags, nullptr, stream);
}

int fp8bq_dispatch_mxfp4_1x32(const void* x, int xtype, int64_t xrows, int64_t cols, int64_t ldx, const int32_t* src,
                              int64_t rows, void* q, int64_t ldq, void* s, int64_t lds, void* qt, int64_t ldqt,
                              void* st, int64_t ldst, int flags, void* workspace, void* stream) {
  return quant("dispatch_mxfp4", x, xtype, xrows, cols, ldx, src, true, rows, q, ldq, s, lds, qt, ldqt, st, ldst,
               flags, workspace, stream);
}

int fp8bq_dequant_mxfp4_1x32(const void* q, int64_t rows, int64_t cols, int64_t ldq, const void* s, int64_t lds,
                             void* y, int ytype, int64_t ldy, void* stream) {
  const char* who = "dequant_mxfp4";
  if (!y) return entry_fail(FP8BQ_E_INVAL, "%s: null pointer", who);
  if (bad_dtype(ytype)) return entry_fail(FP8BQ_E_INVAL, "%s: type must be BF16, FP16 or FP32, got %d", who, ytype);
  if (rows <= 0 || cols <= 0) return entry_fail(FP8BQ_E_INVAL, "%s: rows and cols must be positive", who);
  if (ldy < cols) return entry_fail(FP8BQ_E_INVAL, "%s: ldy < cols", who);
  if (too_large(rows, cols) || ldy > INT64_MAX / 4 / rows)
    return entry_fail(FP8BQ_E_SHAPE, "%s: too large", who);
  if (int e = check_codes(who, "q", q, ldq, s, lds, rows, cols)) return e;
  if (!aligned(y, elem_bytes(ytype))) return entry_fail(FP8BQ_E_ALIGN, "%s: y must be aligned to its element", who);
  if (int e = fp8bq::entry_device()) return e;
  return launched(fp8bq::launch_dequant_mxfp4(static_cast<const uint8_t*>(q), rows, cols, ldq,
                                              static_cast<const uint8_t*>(s), lds, y, ytype, ldy,
                                              reinterpret_cast<hipStream_t>(stream)), who);
}

int fp8bq_gemm_mxfp4(int64_t m, int64_t n, int64_t k, const void* a, int64_t lda, const void* sa, int64_t ldsa,
                     const void* b, int64_t ldb, const void* sb, int64_t ldsb, void* out, int otype, int64_t ldo,
                     void* stream) {
  return gemm("gemm_mxfp4", fp8bq::MX_DENSE, 1, nullptr, m, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, out, otype, ldo,
              stream);
}

int fp8bq_grouped_gemm_mxfp4(int32_t groups, const int32_t* row_off, int64_t m, int64_t n, int64_t k, const void* a,
                             int64_t lda, const void* sa, int64_t ldsa, const void* b, int64_t ldb, const void* sb,
                             int64_t ldsb, void* out, int otype, int64_t ldo, void* stream) {
  return gemm("grouped_gemm_mxfp4", fp8bq::MX_ROWS, groups, row_off, m, n, k, a, lda, sa, ldsa, b, ldb, sb, ldsb, out,
              otype, ldo, stream);
}

int fp8bq_grouped_wgrad_mxfp4(int32_t groups, const int32_t* row_off, int64_t m, int64_t n, int64_t rows, const void* a,
                              int64_t lda, const void* sa, int64_t ldsa, const void* b, int64_t ldb, const void* sb,
                              int64_t ldsb, void* out, int otype, int64_t ldo, void* stream) {
  return gemm("grouped_wgrad_mxfp4", fp8bq::MX_K, groups, row_off, m, n, rows, a, lda, sa, ldsa, b, ldb, sb, ldsb, out,
              otype, ldo, stream);
}

int fp8bq_moe_plan(const int32_t* idx, int64_t tokens, int64_t topk, int64_t ldidx, int32_t groups, int64_t pad,
                   int32_t* counts, int32_t* row_off, int32_t* src, int64_t cap, int32_t* pos, void* workspace,
                   void* stream) {
  const char* who = "moe_plan";
  if (!idx || !counts || !row_off || !src || !pos || !workspace) return entry_fail(FP8BQ_E_INVAL, "%s: null pointer", who);
  if (tokens <= 0 || topk <= 0) return entry_fail(FP8BQ_E_INVAL, "%s: tokens and topk must be positive", who);
  if (ldidx < topk) return entry_fail(FP8BQ_E_INVAL, "%s: ldidx < topk", who);
  if (pad < 1 || pad > 1024) return entry_fail(FP8BQ_E_INVAL, "%s: pad must be 1 .. 1024, got %lld", who, (long long)pad);
  if (groups < 1 || groups > 256) return entry_fail(FP8BQ_E_SHAPE, "%s: groups must be 1 .. 256, got %d", who, groups);
  if (tokens >= kMaxRouted || topk >= kMaxRouted || tokens * topk >= kMaxRouted || cap >= kMaxRouted ||
      ldidx > INT64_MAX / 4 / tokens)
    return entry_fail(FP8BQ_E_SHAPE, "%s: too large", who);
  if (cap < tokens * topk + groups * (pad - 1))
    return entry_fail(FP8BQ_E_INVAL, "%s: cap (%lld) < tokens * topk + groups * (pad - 1)", who, (long long)cap);
  if (!aligned(idx, 4) || !aligned(counts, 4) || !aligned(row_off, 4) || !aligned(src, 4) || !aligned(pos, 4) ||
      !aligned(workspace, 4))
    return entry_fail(FP8BQ_E_ALIGN, "%s: pointers must be 4-byte aligned", who);
  if (int e = fp8bq::entry_device()) return e;
  return launched(fp8bq::launch_moe_plan(idx, (int)tokens, (int)topk, ldidx, groups, (int)pad, counts, row_off, src,
                                         (int)cap, pos, static_cast<int32_t*>(workspace),
                                         reinterpret_cast<hipStream_t>(stream)), who);
}

int fp8bq_moe_balance_workspace_size(int64_t tokens, int64_t experts, int64_t sequences, int64_t* bytes) {
  const char* who = "moe_balance_workspace_size";
  if (!bytes) return entry_fail(FP8BQ_E_INVAL, "%s: null bytes", who);
  if (tokens <= 0 || experts <= 0 || sequences <= 0) return entry_fail(FP8BQ_E_INVAL, "%s: sizes must be positive", who);
  if (experts > 1024 || sequences > 65534 || tokens >= kMaxSide) return entry_fail(FP8BQ_E_SHAPE, "%s: too large", who);
  *bytes = fp8bq::moe_balance_workspace(tokens, experts, sequences);
  return FP8BQ_OK;
}

int fp8bq_moe_balance(const void* logits, int ltype, int64_t tokens, int64_t experts, int64_t ldl, const int32_t* idx,
                      int64_t topk, int64_t ldidx, const int32_t* seq_off, int64_t sequences, int score, float coef,
                      float* loss, int32_t* counts, int32_t* real, void* workspace, void* stream) {
  const char* who = "moe_balance";
  if (!loss || !counts || !real || !workspace) return entry_fail(FP8BQ_E_INVAL, "%s: null pointer", who);
  if (int e = check_balance(who, logits, ltype, tokens, experts, ldl, idx, topk, ldidx, seq_off, sequences, score)) return e;
  if (!aligned(loss, 4) || !aligned(counts, 4) || !aligned(real, 4) || !aligned(workspace, 4))
    return entry_fail(FP8BQ_E_ALIGN, "%s: pointers must be 4-byte aligned", who);
  if (int e = fp8bq::entry_device()) return e;
  return launched(fp8bq::launch_moe_balance(balance_args(logits, tokens, experts, ldl, idx, topk, ldidx, seq_off, sequences, coef),
                                            ltype, score == FP8BQ_SIGMOID, loss, counts, real, workspace,
                                            reinterpret_cast<hipStream_t>(stream)), who);
}

int fp8bq_moe_balance_grad(const float* dloss, const void* logits, int ltype, int64_t tokens, int64_t experts,
                           int64_t ldl, const int32_t* idx, int64_t topk, int64_t ldidx, const int32_t* seq_off,
                           int64_t sequences, int score, float coef, const int32_t* counts, const int32_t* real,
                           void* dlogits, int64_t lddl, void* stream) {
  const char* who = "moe_balance_grad";
  if (!dloss || !counts || !real || !dlogits) return entry_fail(FP8BQ_E_INVAL, "%s: null pointer", who);
  if (int e = check_balance(who, logits, ltype, tokens, experts, ldl, idx, topk, ldidx, seq_off, sequences, score)) return e;
  if (lddl < experts) return entry_fail(FP8BQ_E_INVAL, "%s: lddl < experts", who);
  if (lddl > INT64_MAX / 4 / tokens) return entry_fail(FP8BQ_E_SHAPE, "%s: too large", who);
  if (!aligned(dloss, 4) || !aligned(counts, 4) || !aligned(real, 4) || !aligned(dlogits, elem_bytes(ltype)))
    return entry_fail(FP8BQ_E_ALIGN, "%s: misaligned pointer", who);
  if (int e = fp8bq::entry_device()) return e;
  return launched(fp8bq::launch_moe_balance_grad(balance_args(logits, tokens, experts, ldl, idx, topk, ldidx, seq_off, sequences, coef),
                                                 ltype, score == FP8BQ_SIGMOID, dloss, counts, real, dlogits, lddl,
                                                 reinterpret_cast<hipStream_t>(stream)), who);
}

}  // extern "C"
