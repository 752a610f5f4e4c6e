// Products of a few unquantised rows with MXFP4 weights (weight-only 4 bit):
// out[i][j] = sum_k x[i][k] 2^e[j][k / 32] c[j][k]. Definitions: include/fp8bq.h.
//
// The weight's bytes are the cost (17/32 an element, each read once), so it
// goes from memory straight to registers: lane l of a wave takes 16 bytes, one
// scale group of 32 codes, of weight row l % 16, so that four lanes read 64
// neighbouring bytes of a row. v_cvt_scalef32_pk_bf16_fp4 turns two codes into
// two bf16 with the scale applied, exactly (a code has two significant bits,
// and bf16 the exponents of E8M0 with subnormals), and the products go through
// the bf16 MFMA of 16 x 16 x 32: weights are its 16 rows, x its 16 columns,
// and its 32 positions of K are 8 of each of the four lanes' groups; x is
// fetched in the same order. Sums are fp32. fp16 and fp32 activations are split
// into two and three bf16 terms whose sum is x exactly (11 = 8 + 3 and 24 = 8 +
// 8 + 8 significant bits), each with an MFMA of its own.
#include "../../include/fp8bq.h"
#include "elem.h"
#include "layer.h"
#include "mxfp4_codec.h"

#include <type_traits>

namespace fp8bq {
namespace {

typedef __bf16 v8bf16 __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf16 __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));

template <int T> constexpr int kTerms = T == FP8BQ_BF16 ? 1 : T == FP8BQ_FP16 ? 2 : 3;

// Eight values of x as bf16 terms. Each term is the value's top 8 significant
// bits (cut off, not rounded, so that no finite value becomes infinite); an
// infinity or NaN stays in the first.
template <int T>
__device__ __forceinline__ void split(const Raw8<T>& x, v8bf16 (&t)[kTerms<T>]) {
  if constexpr (T == FP8BQ_BF16) {
    __builtin_memcpy(&t[0], &x, 16);
  } else {
    float v[8];
    values8<T>(x, v);
#pragma unroll
    for (int n = 0; n < kTerms<T>; ++n) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t top[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float& f = v[2 * i + h];
          const uint32_t b = __float_as_uint(f);
          top[h] = b >> 16;
          if ((b & 0x7FFFFFFFu) > 0x7F800000u) top[h] |= 0x40;      // a NaN whose bits are all low
          const float rest = f - __uint_as_float(b & 0xFFFF0000u);
          f = (b & 0x7F800000u) == 0x7F800000u ? 0.f : rest;
        }
        w[i] = top[0] | (top[1] << 16);
      }
      __builtin_memcpy(&t[n], w, 16);
    }
  }
}

__device__ __forceinline__ v8bf16 decode8(uint32_t codes, float scale) {
  const v2bf16 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1),
               c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return v8bf16{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A workgroup makes 16 * NT weight rows' results for 16 * MT rows of x at a
// time; its waves take the chunks of 256 along K in turn and add up their sums
// in LDS, in their order.
template <int T, int MT, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void gemv_kernel(GemvArgs p) {
  using E = typename Elem<T>::type;
  __shared__ v4f part[WAVES][MT * NT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lo = lane & 15, hi = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NT);
  const int chunks = (int)((p.k + 255) / 256);
  const uint8_t *b = p.b, *sb = p.sb;
  int64_t m0 = (int64_t)blockIdx.y * (16 * MT), m1 = min(m0 + 16 * MT, p.m);
  if (p.groups) {
    const int e = blockIdx.y;
    m0 = min(max((int64_t)p.row_off[e], (int64_t)0), p.m);
    m1 = min(max((int64_t)p.row_off[e + 1], m0), p.m);
    b += (int64_t)e * p.n * p.ldb;
    sb += (int64_t)e * chunks * p.ldsb * 8;
  }
  const uint8_t *pb[NT], *ps[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t row = min(n0 + 16 * t + lo, p.n - 1);       // rows past the end repeat the last one
    pb[t] = b + row * p.ldb + 16 * hi;
    ps[t] = sb + row * 8;
  }
  for (; m0 < m1; m0 += 16 * MT) {
    const E* px[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      int64_t row = m0 + 16 * t + lo;
      px[t] = nullptr;
      if (row < m1) {
        if (p.src) row = p.src[row];
        if (row >= 0 && row < p.xrows) px[t] = static_cast<const E*>(p.x) + row * p.ldx + 32 * hi;
      }
    }
    v4f acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int c = wave; c < chunks; c += WAVES) {
      uint4 q[NT][2];
      uint2 s[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        q[t][0] = *reinterpret_cast<const uint4*>(pb[t] + (int64_t)c * 128);
        q[t][1] = *reinterpret_cast<const uint4*>(pb[t] + (int64_t)c * 128 + 64);
        s[t] = *reinterpret_cast<const uint2*>(ps[t] + (int64_t)c * p.ldsb * 8);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float scale[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) scale[t] = mx_scale(((h ? s[t].y : s[t].x) >> (8 * hi)) & 0xFFu);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t col = (int64_t)c * 256 + 128 * h + 8 * j, left = p.k - col - 32 * hi;
          v8bf16 w[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4 v = q[t][h];
            w[t] = decode8(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w, scale[t]);
          }
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            Raw8<T> x{};
            if (px[i]) {
              if (left >= 8) {
                x = load8<T>(px[i] + col);
              } else if (left > 0) {
                E e[8] = {};
#pragma unroll
                for (int z = 0; z < 7; ++z)
                  if (z < left) e[z] = px[i][col + z];
                __builtin_memcpy(&x, e, sizeof(x));
              }
            }
            v8bf16 terms[kTerms<T>];
            split<T>(x, terms);
#pragma unroll
            for (int z = 0; z < kTerms<T>; ++z)
#pragma unroll
              for (int t = 0; t < NT; ++t) acc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[t], terms[z], acc[i][t], 0, 0, 0);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) part[wave][i * NT + j][lane] = acc[i][j];
    __syncthreads();
    // lane's 4 results: rows n0 + 16 j + 4 (lane / 16) .. + 3 of the weight, row m0 + 16 i + lane % 16 of x
    for (int z = wave; z < MT * NT; z += WAVES) {
      v4f v = part[0][z][lane];
#pragma unroll
      for (int u = 1; u < WAVES; ++u) v += part[u][z][lane];
      const int64_t m = m0 + 16 * (z / NT) + lo, n = n0 + 16 * (z % NT) + 4 * hi;
      if (m < m1) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (n + r >= p.n) break;
          const int64_t at = m * p.ldo + n + r;
          if (p.otype == FP8BQ_FP32) static_cast<float*>(p.out)[at] = v[r];
          else if (p.otype == FP8BQ_BF16) static_cast<uint16_t*>(p.out)[at] = Elem<FP8BQ_BF16>::round(v[r]);
          else static_cast<uint16_t*>(p.out)[at] = Elem<FP8BQ_FP16>::round(v[r]);
        }
      }
    }
    __syncthreads();                             // the next rows' sums go to the same place
  }
}

template <int T>
hipError_t run(const GemvArgs& p, hipStream_t st) {
  const dim3 grid((unsigned)((p.n + 15) / 16), (unsigned)(p.groups ? p.groups : (p.m + 15) / 16));
  gemv_kernel<T, 1, 1, 8><<<grid, 512, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemv_mxfp4(const GemvArgs& p, int xtype, hipStream_t st) {
  switch (xtype) {
    case FP8BQ_BF16: return run<FP8BQ_BF16>(p, st);
    case FP8BQ_FP16: return run<FP8BQ_FP16>(p, st);
    default: return run<FP8BQ_FP32>(p, st);
  }
}

}  // namespace fp8bq
