// Internal declarations of the MXFP4 and routing kernels. Nothing here is part
// of the C ABI (include/fp8bq.h is).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxfp4_tiling.h"

namespace fp8bq {

// Launchers. Arguments have been validated by the entry points; each returns
// the hipError_t of its launch. Types are fp8bq_dtype values.

// x [xrows, cols]; with src, row r of the quantised matrix is x[src[r]] (zeros
// where src[r] lies outside), without it xrows == rows. q / qt may be null.
struct MxQuantArgs {
  const void* x;
  int64_t xrows, rows, cols, ldx;
  const int32_t* src;
  uint8_t* q; int64_t ldq;
  uint8_t* s; int64_t lds;
  uint8_t* qt; int64_t ldqt;
  uint8_t* st; int64_t ldst;
};
// ws: null, or (src given, only the row form wanted) xrows * (kMxDispatchSlots +
// 1) words, 16-byte aligned: each x row is then read once and written to every
// row that shows it.
constexpr int kMxDispatchSlots = 8;
hipError_t launch_quant_mxfp4(const MxQuantArgs& a, int xtype, bool nosat, int32_t* ws, hipStream_t stream);
hipError_t launch_dequant_mxfp4(const uint8_t* q, int64_t rows, int64_t cols, int64_t ldq, const uint8_t* s,
                                int64_t lds, void* y, int ytype, int64_t ldy, hipStream_t stream);

// a [m, k], b [n, k] per group. chunks = ceil(k / 256); MX_K: chunks the
// buffers hold, a group's own come from row_off.
struct MxGemmArgs {
  int64_t m, n;
  int chunks;
  const uint8_t* a; int64_t lda;
  const uint8_t* sa; int64_t ldsa;
  const uint8_t* b; int64_t ldb;
  const uint8_t* sb; int64_t ldsb;
  void* out; int64_t ldo;
  int groups;
  const int32_t* row_off;
};
hipError_t launch_gemm_mxfp4(const MxGemmArgs& p, MxMode mode, bool f32_out, hipStream_t stream);

constexpr int kMoePlanMaxBlocks = 256;   // rows of the workspace, one histogram of 256 experts each
hipError_t launch_moe_plan(const int32_t* idx, int tokens, int topk, int64_t ldidx, int groups, int pad,
                           int32_t* counts, int32_t* row_off, int32_t* src, int cap, int32_t* pos, int32_t* ws,
                           hipStream_t stream);

struct MoeBalanceArgs {
  const void* logits; int64_t ldl;
  int64_t tokens;
  int experts, topk;
  const int32_t* idx; int64_t ldidx;
  const int32_t* seq_off;      // null: one sequence of all tokens
  int sequences;
  float coef;
};
int64_t moe_balance_workspace(int64_t tokens, int64_t experts, int64_t sequences);
hipError_t launch_moe_balance(const MoeBalanceArgs& a, int ltype, bool sigmoid, float* loss, int32_t* counts,
                              int32_t* real, void* ws, hipStream_t stream);
hipError_t launch_moe_balance_grad(const MoeBalanceArgs& a, int ltype, bool sigmoid, const float* dloss,
                                   const int32_t* counts, const int32_t* real, void* dlogits, int64_t lddl,
                                   hipStream_t stream);

}  // namespace fp8bq
