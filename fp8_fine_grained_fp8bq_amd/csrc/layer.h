// Internal declarations of the operators around a layer's Linears: the RMS norm,
// tokens to their experts' rows and back, products of a few unquantised rows
// with MXFP4 weights. Nothing here is part of the C ABI (include/fp8bq.h is).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bq {

// Launchers. Arguments have been validated by the entry points; each returns
// the hipError_t of its launch. Types are fp8bq_dtype values.

constexpr int kNormMaxCols = 32768;      // a row stays in the registers of one workgroup

struct NormArgs {
  const void* x; int64_t rows; int cols; int64_t ldx;
  const void* r; int64_t ldr;            // residual, or null
  const void* w; int wtype;
  float eps;
  void* h; int64_t ldh;                  // x + r rounded; null without r
  void* y; int64_t ldy;                  // may be null
  uint8_t* q; int64_t ldq;               // may be null, with s
  float* s; int64_t lds;
  float* rstd;                           // may be null
};
hipError_t launch_rmsnorm(const NormArgs& a, int xtype, bool pow2, hipStream_t stream);

struct NormGradArgs {
  const void* dy; int64_t rows; int cols; int64_t lddy;
  const void* h; int64_t ldh;
  const void* w; int wtype;
  const float* rstd;
  const void* dh; int64_t lddh;          // may be null
  void* dx; int64_t lddx;
  float* dw;
  float* parts;                          // norm_grad_parts(rows, cols) rows of cols sums
};
int64_t norm_grad_parts(int64_t rows, int64_t cols);
hipError_t launch_rmsnorm_grad(const NormGradArgs& a, int xtype, hipStream_t stream);

// Rows [tokens, cols] of `elem` bytes an element to rows pos[t][j] of out; s
// null, or the scales of 1x128 tiles of 8-bit codes with them.
struct MoeDispatchArgs {
  const uint8_t* x; int elem; int64_t tokens, cols, ldx;
  const float* s; int64_t lds;
  const int32_t* pos; int topk;
  const int32_t* src; int64_t rows;
  uint8_t* out; int64_t ldo;
  float* so; int64_t ldso;
};
hipError_t launch_moe_dispatch(const MoeDispatchArgs& a, hipStream_t stream);

struct MoeCombineArgs {
  const void* y; int64_t rows, cols, ldy;
  const int32_t* pos; int64_t tokens; int topk;
  const float* w; int64_t ldw;           // null: every weight 1
  const void* base; int64_t ldb;         // null: nothing besides
  void* out; int64_t ldo;
};
hipError_t launch_moe_combine(const MoeCombineArgs& a, int type, hipStream_t stream);

struct MoeCombineGradArgs {
  const void* dout; int64_t tokens, cols, lddo;
  const void* y; int64_t rows, ldy;
  const int32_t* pos; int topk;
  const float* w; int64_t ldw;
  const int32_t* src;
  void* dy; int64_t lddy;
  float* dw;                             // [tokens, topk]
};
hipError_t launch_moe_combine_grad(const MoeCombineGradArgs& a, int type, hipStream_t stream);

// groups 0: one product of all rows; else rows [row_off[e], row_off[e + 1])
// with weight e. src: row r is x[src[r]] (null: x[r]).
struct GemvArgs {
  int64_t m, n, k;
  const void* x; int64_t xrows, ldx;
  const uint8_t* b; int64_t ldb;
  const uint8_t* sb; int64_t ldsb;
  void* out; int otype; int64_t ldo;
  int groups;
  const int32_t *row_off, *src;
};
hipError_t launch_gemv_mxfp4(const GemvArgs& p, int xtype, hipStream_t stream);

}  // namespace fp8bq
