// Tokens to their experts' rows and back: the rows of a dispatch plan, the
// weighted sum of each token's rows, and its gradient. Definitions:
// include/fp8bq.h. All of it is bound by memory, so each row is read and
// written once: a wave takes a piece of a token's row and visits the token's
// choices (`pos`) with it, instead of each dispatched row fetching its token.
// 8192 tokens of 7168 columns, 8 of 64 experts each, each operator called back to
// back: codes out 105 us (5.2 TB/s), 16-bit rows back 218, its gradient 416.
#include "../../include/fp8bq.h"
#include "elem.h"
#include "lanes.h"
#include "layer.h"

namespace fp8bq {
namespace {

constexpr int kUnit = 8;                 // elements of a lane
constexpr int kChoices = 4;              // choices whose loads are in flight together
                                         // (8: fewer waves; 16384 rows of 2048: 20.7 us, 17.0 with 4)

// Work is numbered in blocks of four waves; workgroups beyond a launch's limit
// take several.
constexpr int64_t kMaxGrid = 1 << 22;
__device__ __forceinline__ int64_t wave_of(int64_t block) { return block * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// A row in units of 16 bytes and, behind the last whole one, single elements:
// item i of a row of `bytes` bytes. Lanes take neighbouring items, so that odd
// sizes end with one more access of a few lanes and not with a loop.
struct Item {
  int64_t at;                            // byte
  bool whole, here;
  __device__ Item(int64_t i, int64_t bytes, int elem) {
    const int64_t units = bytes >> 4;
    whole = i < units;
    at = whole ? i * 16 : units * 16 + (i - units) * elem;
    here = at < bytes;
  }
};
__host__ __device__ int64_t items_of(int64_t bytes, int elem) { return (bytes >> 4) + (bytes & 15) / elem; }

__device__ __forceinline__ void store_element(uint8_t* p, uint32_t v, int elem) {
  if (elem == 1) *p = (uint8_t)v;
  else if (elem == 2) *reinterpret_cast<uint16_t*>(p) = (uint16_t)v;
  else *reinterpret_cast<uint32_t*>(p) = v;
}
__device__ __forceinline__ uint32_t load_element(const uint8_t* p, int elem) {
  if (elem == 1) return *p;
  if (elem == 2) return *reinterpret_cast<const uint16_t*>(p);
  return *reinterpret_cast<const uint32_t*>(p);
}

// Zeros to a row, by one wave.
__device__ __forceinline__ void zero_row(uint8_t* p, int64_t bytes, int elem) {
  const uint4 z = make_uint4(0, 0, 0, 0);
  const int64_t items = items_of(bytes, elem);
  for (int64_t i = threadIdx.x & 63; i < items; i += 64) {
    const Item it(i, bytes, elem);
    if (it.whole) stream_store(p + it.at, z);
    else store_element(p + it.at, 0, elem);
  }
}

// The rows of a plan that no token has (src outside the tokens, but not
// FP8BQ_ROW_UNUSED): four rows a wave.
constexpr int kPadRows = 16;             // of a block
__device__ __forceinline__ void zero_padding(const int32_t* src, int64_t rows, int64_t tokens, uint8_t* out, int64_t row_stride,
                                             int64_t bytes, int elem, int64_t w) {
  for (int64_t r = w * (kPadRows / 4); r < min((w + 1) * (kPadRows / 4), rows); ++r) {
    const int s = src[r];
    if (s != FP8BQ_ROW_UNUSED && (s < 0 || s >= tokens)) zero_row(out + r * row_stride, bytes, elem);
  }
}

// ---------------------------------------------------------------------------
// Dispatch. Blocks [0, copy): pieces of 1 KB of tokens' rows; the next `pad`
// ones: rows without a token; the rest: the scales, 256 rows of 8 tiles each
// (read by row, so that the stores are whole lines).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void dispatch_block(const MoeDispatchArgs& a, int64_t block, int64_t copy, int64_t pad) {
  const int lane = threadIdx.x & 63;
  const int64_t bytes = a.cols * a.elem;
  if (block < copy) {
    const int64_t pieces = (items_of(bytes, a.elem) + 63) / 64;
    const int64_t w = wave_of(block), t = w / pieces;
    const Item it((w - t * pieces) * 64 + lane, bytes, a.elem);
    if (t >= a.tokens || !it.here) return;
    const uint8_t* p = a.x + t * a.ldx * a.elem + it.at;
    const int32_t* pos = a.pos + t * a.topk;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (it.whole) v = load_any<uint4>(p);
    else v.x = load_element(p, a.elem);
    for (int j = 0; j < a.topk; ++j) {
      const int64_t r = pos[j];
      if (r < 0 || r >= a.rows) continue;
      uint8_t* o = a.out + r * a.ldo * a.elem + it.at;
      if (it.whole) stream_store(o, v);
      else store_element(o, v.x, a.elem);
    }
    return;
  }
  if (block < copy + pad) {
    zero_padding(a.src, a.rows, a.tokens, a.out, a.ldo * a.elem, bytes, a.elem, wave_of(block - copy));
    return;
  }
  const int64_t tiles = a.cols / 128, groups = (tiles + 7) / 8;
  const int64_t b = block - copy - pad, r = b / groups * 256 + threadIdx.x, c0 = b % groups * 8;
  if (r >= a.rows) return;
  const int s = a.src[r];
  if (s == FP8BQ_ROW_UNUSED) return;
  for (int64_t c = c0; c < min(c0 + 8, tiles); ++c)
    a.so[c * a.ldso + r] = s >= 0 && s < a.tokens ? a.s[c * a.lds + s] : 0.f;
}
__global__ __launch_bounds__(256) void moe_dispatch_kernel(MoeDispatchArgs a, int64_t copy, int64_t pad, int64_t blocks) {
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) dispatch_block(a, b, copy, pad);
}

// ---------------------------------------------------------------------------
// Combine: out[t] = base[t] + sum_j w[t][j] y[pos[t][j]], in fp32, choices in
// their order, rounded once. A wave takes 512 columns of a token.
// ---------------------------------------------------------------------------
template <int T, int N>
__device__ __forceinline__ void combine(const MoeCombineArgs& a, int64_t t, int64_t col) {
  using E = typename Elem<T>::type;
  using V = Some<T, N>;
  const E* y = static_cast<const E*>(a.y) + col;
  const int32_t* pos = a.pos + t * a.topk;
  const float* gate = a.w ? a.w + t * a.ldw : nullptr;
  float sum[N];
  V base{};
  if (a.base) base = load_any<V>(static_cast<const E*>(a.base) + t * a.ldb + col);
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = Elem<T>::value(base.e[i]);
  for (int j0 = 0; j0 < a.topk; j0 += kChoices) {
    V v[kChoices];
    float g[kChoices];
    bool on[kChoices];
#pragma unroll
    for (int j = 0; j < kChoices; ++j) {
      const int64_t r = j0 + j < a.topk ? pos[j0 + j] : -1;
      on[j] = r >= 0 && r < a.rows;
      g[j] = 1.f;
      v[j] = V{};
      if (on[j]) {
        v[j] = load_any<V>(y + r * a.ldy);
        if (gate) g[j] = gate[j0 + j];
      }
    }
#pragma unroll
    for (int j = 0; j < kChoices; ++j) {
      if (on[j]) {
#pragma unroll
        for (int i = 0; i < N; ++i) sum[i] = __builtin_fmaf(g[j], Elem<T>::value(v[j].e[i]), sum[i]);
      }
    }
  }
  V o;
#pragma unroll
  for (int i = 0; i < N; ++i) o.e[i] = Elem<T>::round(sum[i]);
  stream_store(static_cast<E*>(a.out) + t * a.ldo + col, o);
}

template <int T>
__global__ __launch_bounds__(256) void moe_combine_kernel(MoeCombineArgs a, int64_t blocks) {
  constexpr int N = kUnit;
  const int64_t units = a.cols / N, left = a.cols % N, pieces = (units + left + 63) / 64;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t w = wave_of(b), t = w / pieces, i = (w - t * pieces) * 64 + (threadIdx.x & 63);
    if (t >= a.tokens) return;
    if (i < units) combine<T, N>(a, t, i * N);
    else if (i - units < left) combine<T, 1>(a, t, units * N + i - units);
  }
}

// ---------------------------------------------------------------------------
// Its gradient: dy[pos[t][j]] = w[t][j] dout[t] and dw[t][j] = dout[t] . y[pos[t][j]].
// A block is a token (the dot products need its whole rows), the last ones
// are the rows without one.
// ---------------------------------------------------------------------------
template <int T>
__device__ __forceinline__ void combine_grad(const MoeCombineGradArgs& a, int64_t t, float (&part)[4][kChoices]) {
  using E = typename Elem<T>::type;
  if (t >= a.tokens) {
    zero_padding(a.src, a.rows, a.tokens, static_cast<uint8_t*>(a.dy), a.lddy * Elem<T>::kBytes, a.cols * Elem<T>::kBytes,
                 Elem<T>::kBytes, wave_of(t - a.tokens));
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const E* d = static_cast<const E*>(a.dout) + t * a.lddo;
  const E* y = static_cast<const E*>(a.y);
  E* dy = static_cast<E*>(a.dy);
  const int32_t* pos = a.pos + t * a.topk;
  const int64_t whole = a.cols & ~(int64_t)7, last = whole + threadIdx.x;
  for (int j0 = 0; j0 < a.topk; j0 += kChoices) {
    float dot[kChoices];
    int64_t row[kChoices];
    float g[kChoices];
#pragma unroll
    for (int j = 0; j < kChoices; ++j) {
      dot[j] = 0.f;
      g[j] = 0.f;
      row[j] = j0 + j < a.topk ? pos[j0 + j] : -1;
      if (row[j] >= a.rows) row[j] = -1;
      if (row[j] >= 0) g[j] = a.w[t * a.ldw + j0 + j];
    }
    for (int64_t col = threadIdx.x * 8; col < whole; col += 2048) {
      float f[8];
      Raw8<T> v[kChoices];
      values8<T>(load_any<Raw8<T>>(d + col), f);
#pragma unroll
      for (int j = 0; j < kChoices; ++j) {
        v[j] = Raw8<T>{};
        if (row[j] >= 0) v[j] = load_any<Raw8<T>>(y + row[j] * a.ldy + col);
      }
#pragma unroll
      for (int j = 0; j < kChoices; ++j) {
        if (row[j] >= 0) {
          float o[8], e[8];
          values8<T>(v[j], e);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j] = __builtin_fmaf(f[i], e[i], dot[j]);
            o[i] = g[j] * f[i];
          }
          stream_store(dy + row[j] * a.lddy + col, round8<T>(o));
        }
      }
    }
    if (last < a.cols) {
      const float f = Elem<T>::value(d[last]);
#pragma unroll
      for (int j = 0; j < kChoices; ++j) {
        if (row[j] >= 0) {
          dot[j] = __builtin_fmaf(f, Elem<T>::value(y[row[j] * a.ldy + last]), dot[j]);
          dy[row[j] * a.lddy + last] = Elem<T>::round(g[j] * f);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kChoices; ++j) {
      const float s = wave_sum(dot[j]);
      if (lane == 0) part[wave][j] = s;
    }
    __syncthreads();
    if (threadIdx.x < kChoices && j0 + threadIdx.x < a.topk)
      a.dw[t * a.topk + j0 + threadIdx.x] = part[0][threadIdx.x] + part[1][threadIdx.x] + part[2][threadIdx.x] + part[3][threadIdx.x];
    __syncthreads();
  }
}
template <int T>
__global__ __launch_bounds__(256) void moe_combine_grad_kernel(MoeCombineGradArgs a, int64_t blocks) {
  __shared__ float part[4][kChoices];
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) combine_grad<T>(a, b, part);
}

unsigned grid_of(int64_t blocks) { return (unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid); }

}  // namespace

hipError_t launch_moe_dispatch(const MoeDispatchArgs& a, hipStream_t st) {
  const int64_t copy = (a.tokens * ((items_of(a.cols * a.elem, a.elem) + 63) / 64) + 3) / 4, pad = (a.rows + kPadRows - 1) / kPadRows;
  const int64_t scales = a.s ? (a.rows + 255) / 256 * ((a.cols / 128 + 7) / 8) : 0;
  moe_dispatch_kernel<<<grid_of(copy + pad + scales), 256, 0, st>>>(a, copy, pad, copy + pad + scales);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeCombineArgs& a, int type, hipStream_t st) {
  const int64_t blocks = (a.tokens * ((a.cols / kUnit + a.cols % kUnit + 63) / 64) + 3) / 4;
  switch (type) {
    case FP8BQ_BF16: moe_combine_kernel<FP8BQ_BF16><<<grid_of(blocks), 256, 0, st>>>(a, blocks); break;
    case FP8BQ_FP16: moe_combine_kernel<FP8BQ_FP16><<<grid_of(blocks), 256, 0, st>>>(a, blocks); break;
    default: moe_combine_kernel<FP8BQ_FP32><<<grid_of(blocks), 256, 0, st>>>(a, blocks);
  }
  return hipGetLastError();
}

hipError_t launch_moe_combine_grad(const MoeCombineGradArgs& a, int type, hipStream_t st) {
  const int64_t blocks = a.tokens + (a.rows + kPadRows - 1) / kPadRows;
  switch (type) {
    case FP8BQ_BF16: moe_combine_grad_kernel<FP8BQ_BF16><<<grid_of(blocks), 256, 0, st>>>(a, blocks); break;
    case FP8BQ_FP16: moe_combine_grad_kernel<FP8BQ_FP16><<<grid_of(blocks), 256, 0, st>>>(a, blocks); break;
    default: moe_combine_grad_kernel<FP8BQ_FP32><<<grid_of(blocks), 256, 0, st>>>(a, blocks);
  }
  return hipGetLastError();
}

}  // namespace fp8bq
