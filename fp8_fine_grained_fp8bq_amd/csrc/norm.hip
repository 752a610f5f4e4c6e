// RMS norm of a layer's rows, with the residual's addition before it and the
// 1x128 quantisation of the next FP8 Linear's operand behind it, and its
// gradient. Definitions: include/fp8bq.h.
//
// Forward: h = x + r, y = h w / sqrt(mean h^2 + eps) and per 128 columns
// s = amax|y| / 448, q = E4M3(y / s). A row lives in the registers of its
// lanes as fp32 from the load to the store, so the mean and the scales cost
// no second read: 2 (4 with r) bytes read and 1 to 5 written per 16-bit element.
// Bound by memory. Us, with a residual: 16384 x 7168 with codes and rows 184 to 189
// (5.6 to 5.8 TB/s); 4096 x 7168 with codes 38.6 called back to back on the same
// operands, which a cache then holds in part, 44 on others each time; its gradient,
// dweight's sum included, 46.4 and 54.9.
#include "../../include/fp8bq.h"
#include "elem.h"
#include "fp8_codec.h"
#include "lanes.h"
#include "layer.h"

#include <type_traits>

namespace fp8bq {
namespace {

// ---------------------------------------------------------------------------
// What both directions share: a row belongs to 16 or 64 lanes of a wave (rows
// of up to 128 and 512 columns) or to a whole workgroup; a lane has U units of
// 8 columns, unit u of lane l being columns 8 (l + u L). A tile of 128 columns
// is a unit of 16 neighbouring lanes.
// ---------------------------------------------------------------------------
constexpr int kBlockRow = 0;             // LANES of a row that takes the workgroup

template <int LANES>
__device__ __forceinline__ int lanes_of_row() { return LANES == kBlockRow ? blockDim.x : LANES; }

// Sum over a row's lanes, on each of them. `part` alternates between calls, so
// one barrier a call is enough: the next call but one writes it again.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* part) {
  if constexpr (LANES == 16) return row16_sum(v);
  v = wave_sum(v);
  if constexpr (LANES == kBlockRow) {
    const int waves = blockDim.x >> 6;
    if (waves > 1) {
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
      __syncthreads();
      // lanes of a row of 16 fetch the waves' sums and add them in the same order everywhere
      const int l = threadIdx.x & 15;
      v = row16_sum(l < waves ? part[l] : 0.f);
    }
  }
  return v;
}

// A lane's columns: U units (0: rows of fewer than 8 columns) and, of the up to
// 7 columns behind the last whole unit, one.
template <int LANES, int U>
struct Columns {
  int l, step, full, odd;
  int64_t last;                          // the odd column, or -1
  __device__ Columns(int lane, int cols) : l(lane), step(lanes_of_row<LANES>()), full(cols >> 3), odd(cols & 7) {
    last = l < odd ? (cols & ~7) + l : -1;
  }
  __device__ __forceinline__ bool has(int u) const { return l + u * step < full; }
  __device__ __forceinline__ int64_t col(int u) const { return 8 * (int64_t)(l + u * step); }
  // Where a lane loads from: lanes without the unit share the row's last one.
  __device__ __forceinline__ int64_t source(int u) const { return 8 * (int64_t)min(l + u * step, full - 1); }
};
template <int U> constexpr int kSome = U ? U : 1;

// A lane's weights, of any of the three types.
template <int LANES, int U>
__device__ __forceinline__ void load_weights(const void* w, int wtype, const Columns<LANES, U>& c, float (&v)[kSome<U>][8], float& last) {
  auto get = [&](auto t) {
    constexpr int T = decltype(t)::value;
    const auto* p = static_cast<const typename Elem<T>::type*>(w);
#pragma unroll
    for (int u = 0; u < U; ++u) values8<T>(load8<T>(p + c.source(u)), v[u]);
    last = c.last >= 0 ? Elem<T>::value(p[c.last]) : 0.f;
  };
  if (wtype == FP8BQ_FP32) get(std::integral_constant<int, FP8BQ_FP32>{});
  else if (wtype == FP8BQ_BF16) get(std::integral_constant<int, FP8BQ_BF16>{});
  else get(std::integral_constant<int, FP8BQ_FP16>{});
}

// A lane's elements of the row at p. Every lane loads, and what it has no column
// for is set to zero after: loads under a lane's branch are waited for where the
// branch ends, one after the other (the gradient of 4096 x 7168, called back to
// back: 70 to 84 us, 49.6 without the branches when they went).
template <int T, int U>
struct Row {
  Raw8<T> unit[kSome<U>];
  typename Elem<T>::type last;
  template <int LANES>
  __device__ __forceinline__ void load(const void* base, int64_t at, const Columns<LANES, U>& c) {
    const auto* p = static_cast<const typename Elem<T>::type*>(base) + at;
    last = {};
    if (c.odd) last = p[max(c.last, (int64_t)0)];              // uniform
#pragma unroll
    for (int u = 0; u < U; ++u) unit[u] = load8<T>(p + c.source(u));
  }
  template <int LANES>
  __device__ __forceinline__ void clear(const Columns<LANES, U>& c, bool here = true) {
    if (!here || c.last < 0) last = {};
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (!here || !c.has(u)) unit[u] = Raw8<T>{};
  }
};

constexpr float kMinNormal = 0x1p-126f;

// The scale of a tile whose largest magnitude is amax (as fp8_codec.h has it
// for bf16 magnitudes): s = fl32(amax / 448), or the power of two.
__device__ __forceinline__ TileScale tile_scale(float amax, bool pow2) {
  TileScale t;
  if (pow2) {
    const uint32_t b = __float_as_uint(amax);
    const int k = max(-127, min(127, (int)(b >> 23) - 135 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0)));
    t.s = k >= -126 ? __uint_as_float((uint32_t)(k + 127) << 23) : __uint_as_float(0x00400000u);
    t.y = __uint_as_float((uint32_t)(127 - k) << 23);
    t.fast = true;
    return t;
  }
  t.s = amax / kFmax;
  t.fast = t.s == 0.f || t.s >= kFastScaleMin;
  t.y = t.fast && t.s != 0.f ? 1.0f / t.s : 0.f;
  return t;
}

// ---------------------------------------------------------------------------
// Forward. Workgroups walk over the rows.
// ---------------------------------------------------------------------------
template <int T, int LANES, int U, int THREADS, bool RES>
__global__ __launch_bounds__(THREADS) void rmsnorm_kernel(NormArgs a, bool pow2) {
  using E = typename Elem<T>::type;
  __shared__ float part[2][16];
  const int per_block = LANES == kBlockRow ? 1 : 256 / LANES;
  const int sub = LANES == kBlockRow ? 0 : threadIdx.x / LANES;
  const Columns<LANES, U> c(LANES == kBlockRow ? threadIdx.x : threadIdx.x % LANES, a.cols);
  float w[kSome<U>][8], wlast;
  load_weights(a.w, a.wtype, c, w, wlast);

  int turn = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * per_block; row0 < a.rows; row0 += (int64_t)gridDim.x * per_block, turn ^= 1) {
    const int64_t row = row0 + sub;
    const bool here = row < a.rows;              // (a whole workgroup's row always is)
    const int64_t from = here ? row : a.rows - 1;
    Row<T, U> x, r;
    x.load(a.x, from * a.ldx, c);
    if constexpr (RES) r.load(a.r, from * a.ldr, c);
    x.clear(c);
    if constexpr (RES) r.clear(c);
    float v[kSome<U>][8], vlast = Elem<T>::value(x.last);
    if constexpr (RES) {
      vlast += Elem<T>::value(r.last);
      if (here && c.last >= 0) static_cast<E*>(a.h)[row * a.ldh + c.last] = Elem<T>::round(vlast);
    }
    float ss = vlast * vlast;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      values8<T>(x.unit[u], v[u]);
      if constexpr (RES) {
        float o[8];
        values8<T>(r.unit[u], o);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] += o[i];
        if (here && c.has(u)) stream_store(static_cast<E*>(a.h) + row * a.ldh + c.col(u), round8<T>(v[u]));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(v[u][i], v[u][i], ss);
    }
    const float rstd = 1.0f / __builtin_sqrtf(row_sum<LANES>(ss, part[turn]) / (float)a.cols + a.eps);
    if (a.rstd && here && c.l == 0) a.rstd[row] = rstd;
    if (a.y && here && c.last >= 0) static_cast<E*>(a.y)[row * a.ldy + c.last] = Elem<T>::round(vlast * rstd * wlast);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool mine = here && c.has(u);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = v[u][i] * rstd * w[u][i];
      TileScale t;
      uint2 e;
      auto encode = [&](const float (&f)[8], auto p2) {
        e.x = encode4<decltype(p2)::value>(f[0], f[1], f[2], f[3], t);
        e.y = encode4<decltype(p2)::value>(f[4], f[5], f[6], f[7], t);
      };
      auto amax = [](const float (&f)[8]) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
        return row16_max(m);
      };
      if (a.q) {                                 // cols is a multiple of 128: a tile's 16 lanes have the unit or not together
        if (pow2) {
          t = tile_scale(amax(y), true);
          encode(y, std::true_type{});
        } else {
          // rstd is a factor of the whole tile: it goes into the scale, and the codes come from h w, off by the roundings
          // of that product, of the tile's amax / 448 and of the quotient only. They come from y where h w may have
          // underflowed or has overflowed, and where the scale is subnormal, with which they go as it is rounded.
          float hw[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) hw[i] = v[u][i] * w[u][i];
          t = tile_scale(amax(hw), false);
          if (t.s >= kFastScaleMin && t.s < INFINITY && t.s * rstd >= kMinNormal) {
            encode(hw, std::false_type{});
            t.s *= rstd;
          } else {
            t = tile_scale(amax(y), false);
            const float most = kFmax * t.s;      // a subnormal scale may be rounded off by a third: codes end at 448
            float ends[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) ends[i] = fabsf(y[i]) > most ? __builtin_copysignf(most, y[i]) : y[i];
            encode(ends, std::false_type{});
          }
        }
      }
      if (a.y && mine) stream_store(static_cast<E*>(a.y) + row * a.ldy + c.col(u), round8<T>(y));
      if (a.q && mine) {
        *reinterpret_cast<uint2*>(a.q + row * a.ldq + c.col(u)) = e;
        if ((c.l & 15) == 0) a.s[(c.col(u) >> 7) * a.lds + row] = t.s;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Gradient. With xh = h rstd and g = dy w: dx = rstd (g - xh mean(g xh)) + dh,
// dw = sum over the rows of dy xh. The lanes of a row walk over rows, keep their
// columns' share of dw in registers, and a workgroup writes its share out at its
// end; a second kernel adds the workgroups' shares in their order. Bound by
// memory: 6 bytes (8 with dh) a 16-bit element.
// ---------------------------------------------------------------------------
template <int T, int LANES, int U, int THREADS, bool DH>
__global__ __launch_bounds__(THREADS) void rmsnorm_grad_kernel(NormGradArgs a) {
  using E = typename Elem<T>::type;
  __shared__ float part[2][16];
  const Columns<LANES, U> c(LANES == kBlockRow ? threadIdx.x : threadIdx.x % LANES, a.cols);
  const int group = LANES == kBlockRow ? blockIdx.x : blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  const int64_t groups = LANES == kBlockRow ? gridDim.x : (int64_t)gridDim.x * (256 / LANES);
  const int64_t turns = (a.rows + groups - 1) / groups;      // the same for every group: barriers and lane sums in step
  float w[kSome<U>][8], dw[kSome<U>][8], wlast, dwlast = 0.f;
  load_weights(a.w, a.wtype, c, w, wlast);
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[u][i] = 0.f;
  for (int64_t k = 0; k < turns; ++k) {
    const int64_t row = k * groups + group;
    const bool here = row < a.rows;
    const int64_t from = here ? row : a.rows - 1;
    Row<T, U> y, x, r;
    y.load(a.dy, from * a.lddy, c);
    x.load(a.h, from * a.ldh, c);
    if constexpr (DH) r.load(a.dh, from * a.lddh, c);
    const float rstd = a.rstd[from];
    y.clear(c, here);
    x.clear(c, here);
    const float dylast = Elem<T>::value(y.last), xhlast = Elem<T>::value(x.last) * rstd;
    float dot = dylast * wlast * xhlast;
    dwlast = __builtin_fmaf(dylast, xhlast, dwlast);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float dy[8], h[8];
      values8<T>(y.unit[u], dy);
      values8<T>(x.unit[u], h);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = h[i] * rstd;
        dot = __builtin_fmaf(dy[i] * w[u][i], xh, dot);
        dw[u][i] = __builtin_fmaf(dy[i], xh, dw[u][i]);
      }
    }
    const float mean = row_sum<LANES>(dot, part[k & 1]) / (float)a.cols;
    E* out = static_cast<E*>(a.dx) + row * a.lddx;
    if (here && c.last >= 0) {
      float dx = rstd * __builtin_fmaf(-xhlast, mean, dylast * wlast);
      if constexpr (DH) dx += Elem<T>::value(r.last);
      out[c.last] = Elem<T>::round(dx);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (here && c.has(u)) {
        float dy[8], h[8], d[8];
        values8<T>(y.unit[u], dy);
        values8<T>(x.unit[u], h);
        if constexpr (DH) values8<T>(r.unit[u], d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float dx = rstd * __builtin_fmaf(-(h[i] * rstd), mean, dy[i] * w[u][i]);
          d[i] = DH ? dx + d[i] : dx;
        }
        stream_store(out + c.col(u), round8<T>(d));
      }
    }
  }
  // the workgroup's share: of the groups in it, in their order
  float* out = gridDim.x == 1 ? a.dw : a.parts + (int64_t)blockIdx.x * a.cols;
  if constexpr (LANES == kBlockRow) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c.has(u)) __builtin_memcpy(out + c.col(u), dw[u], sizeof(dw[u]));
    if (c.last >= 0) out[c.last] = dwlast;
  } else {
    constexpr int kCols = LANES * 8;               // at most this many
    __shared__ float share[256 / LANES][kCols];
    float* mine = share[threadIdx.x / LANES];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c.has(u)) __builtin_memcpy(mine + c.col(u), dw[u], sizeof(dw[u]));
    if (c.last >= 0) mine[c.last] = dwlast;
    __syncthreads();
    for (int col = threadIdx.x; col < a.cols; col += 256) {
      float v = 0.f;
#pragma unroll
      for (int g = 0; g < 256 / LANES; ++g) v += share[g][col];
      out[col] = v;
    }
  }
}

// dw: 64 columns a workgroup, its 16 waves each adding every 16th row of sums.
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(const float* parts, int rows, int cols, float* dw) {
  __shared__ float sum[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  float v = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (int r = wave; r < rows; r += 16) v += parts[(int64_t)r * cols + col];
  }
  sum[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && col < cols) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sum[i][lane];
    dw[col] = t;
  }
}

// How a row of `cols` columns is dealt: f(lanes, units, bound on the threads of
// a workgroup, threads), the first three as constants. Up to 512 threads keep
// 256 registers each, so that rows need no scratch memory up to 16384 columns
// (24 bytes a lane for the fp32 gradient with dh above 8192). Up to 1024 threads
// have 128, and wider rows keep 48 to 80 bytes there with a residual and 412 to
// 544 in the gradient: us for bf16 with a residual and dh, 1792 rows of 16384
// 46.3 and 55.2, 1778 of 16512 59.5 and 236, 896 of 32768 59.4 and 224.
template <class F>
void with_shape(int64_t cols, F&& f) {
  using std::integral_constant;
  const int64_t units = cols / 8;
  auto threads = [&](int u) { return (int)((units + 64 * u - 1) / (64 * u) * 64); };
  if (cols < 8) f(integral_constant<int, 16>{}, integral_constant<int, 0>{}, integral_constant<int, 256>{}, 256);
  else if (cols <= 128) f(integral_constant<int, 16>{}, integral_constant<int, 1>{}, integral_constant<int, 256>{}, 256);
  else if (cols <= 512) f(integral_constant<int, 64>{}, integral_constant<int, 1>{}, integral_constant<int, 256>{}, 256);
  else if (units <= 512) f(integral_constant<int, kBlockRow>{}, integral_constant<int, 1>{}, integral_constant<int, 512>{}, threads(1));
  else if (units <= 1024) f(integral_constant<int, kBlockRow>{}, integral_constant<int, 2>{}, integral_constant<int, 512>{}, threads(2));
  else if (units <= 2048) f(integral_constant<int, kBlockRow>{}, integral_constant<int, 4>{}, integral_constant<int, 512>{}, threads(4));
  else f(integral_constant<int, kBlockRow>{}, integral_constant<int, 4>{}, integral_constant<int, 1024>{}, threads(4));
}

template <int T, bool RES>
hipError_t forward(const NormArgs& a, bool pow2, hipStream_t st) {
  with_shape(a.cols, [&](auto lanes, auto units, auto bound, int threads) {
    const int64_t per_block = lanes == kBlockRow ? 1 : 256 / (lanes == kBlockRow ? 1 : lanes);
    const int64_t blocks = (a.rows + per_block - 1) / per_block;
    rmsnorm_kernel<T, decltype(lanes)::value, decltype(units)::value, decltype(bound)::value, RES>
        <<<(unsigned)(blocks < (1 << 22) ? blocks : 1 << 22), threads, 0, st>>>(a, pow2);
  });
  return hipGetLastError();
}

// Workgroups of the gradient, of which each leaves a row of sums: enough to fill
// the chip, few enough that their sums are a small part of the traffic. Us with
// 256 / 512 / 1024 where a row takes a workgroup: 2048 x 16384 54.8 / 62.4 / 75.5,
// 4096 x 7168 49.0 / 49.5 to 52.8 / 57.1, 16384 x 2048 83 / 55.5 / 49.7. At least
// two rows each (333 x 2048 fp32: 7.4 us, 8.7 with one).
int grad_blocks(int64_t rows, int64_t cols) {
  int64_t most = cols > 8192 ? 256 : cols > 2048 ? 512 : 1024;
  if (cols <= 128) rows = (rows + 15) / 16;
  else if (cols <= 512) rows = (rows + 3) / 4;
  most = most < (rows + 1) / 2 ? most : (rows + 1) / 2;
  return (int)most;
}

template <int T, bool DH>
hipError_t gradient(const NormGradArgs& a, hipStream_t st) {
  const int blocks = grad_blocks(a.rows, a.cols);
  with_shape(a.cols, [&](auto lanes, auto units, auto bound, int threads) {
    rmsnorm_grad_kernel<T, decltype(lanes)::value, decltype(units)::value, decltype(bound)::value, DH><<<blocks, threads, 0, st>>>(a);
  });
  if (hipError_t e = hipGetLastError(); e != hipSuccess || blocks == 1) return e;
  rmsnorm_dw_kernel<<<(a.cols + 63) / 64, 1024, 0, st>>>(a.parts, blocks, a.cols, a.dw);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, int xtype, bool pow2, hipStream_t st) {
  switch (xtype) {
    case FP8BQ_BF16: return a.r ? forward<FP8BQ_BF16, true>(a, pow2, st) : forward<FP8BQ_BF16, false>(a, pow2, st);
    case FP8BQ_FP16: return a.r ? forward<FP8BQ_FP16, true>(a, pow2, st) : forward<FP8BQ_FP16, false>(a, pow2, st);
    default: return a.r ? forward<FP8BQ_FP32, true>(a, pow2, st) : forward<FP8BQ_FP32, false>(a, pow2, st);
  }
}

int64_t norm_grad_parts(int64_t rows, int64_t cols) { return grad_blocks(rows, cols); }

hipError_t launch_rmsnorm_grad(const NormGradArgs& a, int xtype, hipStream_t st) {
  switch (xtype) {
    case FP8BQ_BF16: return a.dh ? gradient<FP8BQ_BF16, true>(a, st) : gradient<FP8BQ_BF16, false>(a, st);
    case FP8BQ_FP16: return a.dh ? gradient<FP8BQ_FP16, true>(a, st) : gradient<FP8BQ_FP16, false>(a, st);
    default: return a.dh ? gradient<FP8BQ_FP32, true>(a, st) : gradient<FP8BQ_FP32, false>(a, st);
  }
}

}  // namespace fp8bq
