// Products of a few unquantised rows with MXFP4 weights (weight-only 4 bit):
// out[i][j] = sum_k x[i][k] 2^e[j][k / 32] c[j][k]. Definitions: include/fp8bq.h.
//
// The weight's bytes are the cost (17/32 an element, each read once for up to 16
// rows), so it goes from memory straight to registers: lane l of a wave takes 16
// bytes, one scale group of 32 codes, of weight row l % 16, so that four lanes
// read 64 neighbouring bytes of a row. v_cvt_scalef32_pk_bf16_fp4 turns two codes
// into two bf16 with the scale applied, exactly (a code has two significant bits,
// and bf16 the exponents of E8M0 with subnormals, but for products of 2^128 and
// more, which become infinite), and the products go through the bf16 MFMA of
// 16 x 16 x 32: weights are its 16 rows, x its 16 columns, and its 32 positions of
// K are 8 of each of the four lanes' groups; x is fetched in the same order. Sums
// are fp32. fp32 activations are split into three bf16 terms whose sum is x exactly
// (24 = 8 + 8 + 8 significant bits) down to bf16's 2^-133, each with an MFMA of its
// own. fp16 ones meet weights decoded to fp16 where the scales of all lanes allow
// that exactly, as those of a model's weights do (all but those of tiles of zeros);
// else they are split into two bf16 terms (11 = 8 + 3 bits).
//
// What bounds it: the weight's bytes, once enough loads are in flight; for 9 to 16
// rows also x, whose chunk takes 32 registers a lane where a weight tile's takes
// 10, so that fewer are in flight. One row of 18432 x 7168 (70 MB) takes 14.4 us,
// 15.8 with the weight out of the caches; the same loads alone take 15. What it
// took (us, the same product): x loaded by the lanes that use it 20 (a load for
// every lane of the MFMA's 16 columns fills the 64 bytes a cycle of the CU's
// vector cache), x held in registers over many weight tiles 30 and x staged for a
// workgroup with a barrier a step 19 (both wait for memory in step), branches
// around the loads 27 to 40.
#include "../../include/fp8bq.h"
#include "elem.h"
#include "layer.h"
#include "mxfp4_codec.h"

#include <type_traits>

namespace fp8bq {
namespace {

typedef __bf16 v8bf16 __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf16 __attribute__((ext_vector_type(2)));
typedef _Float16 v8f16 __attribute__((ext_vector_type(8)));
typedef _Float16 v2f16 __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));

// bf16 terms of an element of x.
template <int T> constexpr int kTerms = T == FP8BQ_BF16 ? 1 : T == FP8BQ_FP16 ? 2 : 3;

// Eight values of x as bf16 terms. Each term is the top 8 significant bits of
// what the ones before it leave (cut off, not rounded, so that no finite value
// becomes infinite); an infinity or NaN stays in the first, the others are then
// zero. SPECIAL: there may be one.
template <int T, bool SPECIAL>
__device__ __forceinline__ void split(const float (&x)[8], v8bf16 (&t)[kTerms<T>]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = x[i];
#pragma unroll
  for (int n = 0; n < kTerms<T>; ++n) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t b[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float& f = v[2 * i + h];
        b[h] = __float_as_uint(f);
        const float rest = f - __uint_as_float(b[h] & 0xFFFF0000u);
        f = SPECIAL && (b[h] & 0x7F800000u) == 0x7F800000u ? 0.f : rest;
        if (SPECIAL && (b[h] & 0x7FFFFFFFu) > 0x7F800000u) b[h] |= 0x400000u;      // a NaN whose bits are all low
      }
      w[i] = (b[0] >> 16) | (b[1] & 0xFFFF0000u);
    }
    __builtin_memcpy(&t[n], w, 16);
  }
}
template <int T>
__device__ __forceinline__ void terms_of(const Raw8<T>& x, v8bf16 (&t)[kTerms<T>]) {
  if constexpr (T == FP8BQ_BF16) {
    __builtin_memcpy(&t[0], &x, 16);
  } else {
    float v[8];
    values8<T>(x, v);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    if (__any(top >= 0x7F800000u)) split<T, true>(v, t);
    else split<T, false>(v, t);
  }
}

__device__ __forceinline__ v8bf16 decode8(uint32_t codes, float scale) {
  const v2bf16 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1),
               c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return v8bf16{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ v8f16 decode8_f16(uint32_t codes, float scale) {
  const v2f16 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 1),
              c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 3);
  return v8f16{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// fp16 holds a code times 2^e exactly for e from -23 (half of it is the
// smallest subnormal) to 13 (6 * 2^13 = 49152): scale bytes 104 to 140.
__device__ __forceinline__ bool fits_f16(uint32_t byte) { return byte - 104u <= 36u; }

template <int T>
__device__ __forceinline__ void store4(void* out, int64_t at, int n, v4f v) {
  using E = typename Elem<T>::type;
  E e[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) e[r] = Elem<T>::round(v[r]);
  E* p = static_cast<E*>(out) + at;
  if (n >= 4) {
    __builtin_memcpy(p, e, sizeof(e));
  } else {
#pragma unroll
    for (int r = 0; r < 3; ++r)
      if (r < n) p[r] = e[r];
  }
}

// ---------------------------------------------------------------------------
// Up to 2 P rows of x (P = 1 .. 8): no barrier until the end. The waves of a
// workgroup have the same 16 * NT weight rows and take the chunks of 256 along K
// in turn; each passes its chunk of x through LDS of its own, where the lanes of
// rows that are not there share those of the last one (a load for every lane
// would cost the CU's 64 bytes a cycle of the vector cache 16 times for one row).
// ---------------------------------------------------------------------------
template <int T, int P, int NT>
struct Few {
  using E = typename Elem<T>::type;
  static constexpr int kPlanes = T == FP8BQ_FP32 ? 3 : 1;
  static constexpr int kRows = 2 * P;
  struct Shared { uint4 x[kPlanes][kRows * 32]; };             // of one wave: [step][lane / 16][row]
  struct Stage {
    Raw8<T> x[P];
    uint4 q[NT][2];
    uint2 s[NT];
  };
  const GemvArgs& p;
  Shared& sh;
  int lane, lo, hi;
  const uint8_t *b, *sb;                 // of the workgroup's first weight row
  uint32_t ob[NT], os[NT];
  const E* px[P];                        // what this lane loads of a chunk

  // Unit u (8 elements) of row r: step z of the MFMAs takes it to lane 16 h + r.
  static __device__ __forceinline__ int slot(int r, int z, int h) {
    const int at = (z * 4 + h) * kRows + r;
    static_assert(kRows < 8 || kRows % 8 == 0, "the places of a unit's rows are whole groups of 8");
    return kRows >= 8 ? at ^ ((z & 3) + 4 * (h & 1)) : at;     // neighbouring units of a row to different banks
  }
  __device__ __forceinline__ void load_codes(Stage& t, int c) const {
    const uint8_t *bc = b + (int64_t)c * 128, *sc = sb + (int64_t)c * p.ldsb * 8;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      t.q[i][0] = *reinterpret_cast<const uint4*>(bc + ob[i]);
      t.q[i][1] = *reinterpret_cast<const uint4*>(bc + ob[i] + 64);
      t.s[i] = *reinterpret_cast<const uint2*>(sc + os[i]);
    }
  }
  // Chunk c, which px stands `ahead` chunks before. Nothing here or in the loop
  // around it branches: behind a branch the compiler waits for every load in
  // flight.
  __device__ __forceinline__ void load(Stage& t, int c, int ahead = 0) const {
#pragma unroll
    for (int i = 0; i < P; ++i) t.x[i] = load8<T>(px[i] + ahead * 256);
    load_codes(t, c);
  }
  __device__ __forceinline__ void advance(int chunks) {
#pragma unroll
    for (int i = 0; i < P; ++i) px[i] += chunks * 256;
  }
  __device__ __forceinline__ void load_last(Stage& t, int c) const {
    const int left = (int)(p.k - (int64_t)c * 256) - 8 * (lane & 31);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      E e[8] = {};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) e[j] = px[i][j];
      __builtin_memcpy(&t.x[i], e, sizeof(e));
    }
    load_codes(t, c);
  }
  __device__ __forceinline__ void use(const Stage& t, v4f (&acc)[NT]) const {
    const int u = lane & 31;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int at = slot(2 * i + (lane >> 5), (u >> 4) * 4 + (u & 3), (u >> 2) & 3);
      if constexpr (kPlanes == 1) {
        __builtin_memcpy(&sh.x[0][at], &t.x[i], 16);
      } else {
        v8bf16 terms[kTerms<T>];
        terms_of<T>(t.x[i], terms);
#pragma unroll
        for (int n = 0; n < kPlanes; ++n) __builtin_memcpy(&sh.x[n][at], &terms[n], 16);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");     // the wave's LDS accesses stay in this order
    bool fits = true;
    uint32_t byte[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      byte[i][0] = (t.s[i].x >> (8 * hi)) & 0xFFu;
      byte[i][1] = (t.s[i].y >> (8 * hi)) & 0xFFu;
      fits = fits && fits_f16(byte[i][0]) && fits_f16(byte[i][1]);
    }
    const bool f16 = T == FP8BQ_FP16 && __all(fits);
    const int r = min(lo, kRows - 1);
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      uint4 x[kPlanes];
#pragma unroll
      for (int n = 0; n < kPlanes; ++n) x[n] = sh.x[n][slot(r, z, hi)];
      auto code = [&](int i) {
        const uint4 v = t.q[i][z >> 2];
        return (z & 3) == 0 ? v.x : (z & 3) == 1 ? v.y : (z & 3) == 2 ? v.z : v.w;
      };
      if (f16) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(decode8_f16(code(i), mx_scale(byte[i][z >> 2])), __builtin_bit_cast(v8f16, x[0]), acc[i], 0, 0, 0);
        continue;
      }
      v8bf16 terms[kTerms<T>];
      if constexpr (T == FP8BQ_FP16) {
        terms_of<T>(__builtin_bit_cast(Raw8<T>, x[0]), terms);
      } else {
#pragma unroll
        for (int n = 0; n < kPlanes; ++n) terms[n] = __builtin_bit_cast(v8bf16, x[n]);
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const v8bf16 w = decode8(code(i), mx_scale(byte[i][z >> 2]));
#pragma unroll
        for (int n = 0; n < kTerms<T>; ++n) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, terms[n], acc[i], 0, 0, 0);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
};

__device__ __forceinline__ void store_result(const GemvArgs& p, int64_t m, int64_t n, v4f v) {
  if (n >= p.n) return;
  if (p.src && !(p.src[m] >= 0 && p.src[m] < p.xrows)) v = v4f{0.f, 0.f, 0.f, 0.f};
  const int left = (int)min((int64_t)4, p.n - n);
  if (p.otype == FP8BQ_FP32) store4<FP8BQ_FP32>(p.out, m * p.ldo + n, left, v);
  else if (p.otype == FP8BQ_BF16) store4<FP8BQ_BF16>(p.out, m * p.ldo + n, left, v);
  else store4<FP8BQ_FP16>(p.out, m * p.ldo + n, left, v);
}

// Rows m0 .. m1 of the result, 2 P at a time, for weight rows n0 .. n0 + 16 NT.
// lds: of WAVES * (sizeof(Few::Shared) + NT KB).
template <int T, int P, int NT, int WAVES>
__device__ __forceinline__ void few_rows(const GemvArgs& p, const uint8_t* b, const uint8_t* sb, int64_t n0, int64_t m0, int64_t m1, char* lds) {
  using F = Few<T, P, NT>;
  using E = typename Elem<T>::type;
  const int whole = (int)(p.k / 256);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  v4f* part = reinterpret_cast<v4f*>(lds);       // [wave][tile][lane]
  F f{p, reinterpret_cast<typename F::Shared*>(lds + WAVES * NT * 1024)[wave], lane, lane & 15, lane >> 4, b + n0 * p.ldb, sb + n0 * 8};
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const uint32_t r = (uint32_t)min((int64_t)(16 * i + f.lo), p.n - 1 - n0);       // rows past the end repeat the last one
    f.ob[i] = r * (uint32_t)p.ldb + 16 * f.hi;
    f.os[i] = r * 8;
  }
  for (; m0 < m1; m0 += F::kRows) {
#pragma unroll
    for (int i = 0; i < P; ++i) {        // rows past the end repeat the last one, rows of zeros take any
      const int64_t r = min(m0 + 2 * i + (lane >> 5), m1 - 1), x = p.src ? p.src[r] : r;
      f.px[i] = static_cast<const E*>(p.x) + (x >= 0 && x < p.xrows ? x : 0) * p.ldx + 8 * (lane & 31) + wave * 256;
    }
    v4f acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
    typename F::Stage st[2];
    int c = wave;
    if (c < whole) {
      f.load(st[0], c);
      for (; c + WAVES < whole; c += 2 * WAVES) {
        f.load(st[1], c + WAVES, WAVES);
        f.use(st[0], acc);
        const int next = min(c + 2 * WAVES, whole - 1);        // the last load may be one that nobody uses
        f.advance(next - c);
        f.load(st[0], next);
        f.use(st[1], acc);
      }
      if (c < whole) {
        f.use(st[0], acc);
        f.advance(WAVES);
        c += WAVES;
      } else {
        f.advance(c - (whole - 1));
      }
    }
    if (c == whole && p.k % 256) {       // the chunk that k ends in
      f.load_last(st[0], c);
      f.use(st[0], acc);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) part[(wave * NT + i) * 64 + lane] = acc[i];
    __syncthreads();
    for (int i = wave; i < NT; i += WAVES) {
      v4f v = part[i * 64 + lane];
#pragma unroll
      for (int u = 1; u < WAVES; ++u) v += part[(u * NT + i) * 64 + lane];
      if (f.lo < F::kRows && m0 + f.lo < m1) store_result(p, m0 + f.lo, n0 + 16 * i + 4 * f.hi, v);
    }
    __syncthreads();                     // the next rows' sums go to the same place
  }
}

// One product: P by the number of rows.
template <int T, int P, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void gemv_kernel(GemvArgs p) {
  __shared__ __align__(16) char lds[WAVES * (sizeof(typename Few<T, P, NT>::Shared) + NT * 1024)];
  const int64_t m0 = (int64_t)blockIdx.y * (2 * P);
  few_rows<T, P, NT, WAVES>(p, p.b, p.sb, (int64_t)blockIdx.x * (16 * NT), m0, min(m0 + 2 * P, p.m), lds);
}

// Experts: only here are the numbers of their rows known.
template <int T, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void grouped_gemv_kernel(GemvArgs p) {
  __shared__ __align__(16) char lds[WAVES * (sizeof(typename Few<T, 8, NT>::Shared) + NT * 1024)];
  const int e = blockIdx.y;
  const int64_t m0 = min(max((int64_t)p.row_off[e], (int64_t)0), p.m), m1 = min(max((int64_t)p.row_off[e + 1], m0), p.m);
  const uint8_t *b = p.b + (int64_t)e * p.n * p.ldb, *sb = p.sb + (int64_t)e * ((p.k + 255) / 256) * p.ldsb * 8;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NT);
  if (m1 - m0 <= 2) few_rows<T, 1, NT, WAVES>(p, b, sb, n0, m0, m1, lds);
  else if (m1 - m0 <= 4) few_rows<T, 2, NT, WAVES>(p, b, sb, n0, m0, m1, lds);
  else few_rows<T, 8, NT, WAVES>(p, b, sb, n0, m0, m1, lds);
}

template <int T, int P, int NT>
void launch_dense(const GemvArgs& p, hipStream_t st) {
  const dim3 grid((unsigned)((p.n + 16 * NT - 1) / (16 * NT)), (unsigned)((p.m + 2 * P - 1) / (2 * P)));
  gemv_kernel<T, P, NT, 4><<<grid, 256, 0, st>>>(p);
}
// Tiles a wave, from 3 rows on: x is loaded once for all tiles of a workgroup and
// costs about as much as one of them, and workgroups run in rounds of 256, one a
// CU; so the number with the least rounds * (tiles + 1). Us with one to five
// tiles, weights out of the caches: 16 rows of bf16, k = 4096, n = 8192 10.5 / 8.3 /
// 9.6 / 11.9 / 12.3, n = 20480 20.5 / 17.7 / 16.1 / 19.7 / 13.6, n = 24576 24.3 /
// 18.6 / 16.9 / 20.3 / 21.7; 4 rows of 18432 x 7168 18.8 / 18.5 / 17.6 / 21.6 / 15.7.
// From n = 12289 to 16384 it is four, 4% from five at most for bf16 (n = 13312 16.8 / 13.1 /
// 15.8 / 12.5 / 12.9, k = 7168 24.9 / 18.9 / 22.1 / 17.7 / 18.1) and a tenth less for fp16
// (25.7 / 20.1 / 24.2 / 18.8 / 20.9). One and two rows differ by 1% where five tiles do
// best (15.8 / 15.6) and take one. fp32 with more than 8 rows has registers for three
// (16 rows, k = 7168, one to three tiles: n = 2048 20.1 / 21.8 / 24.7, n = 7168 38 / 22 /
// 25, n = 18432 91 / 61 / 48). Four tiles of bf16 for 16 rows and five of fp32 for 8
// keep 16 bytes a lane in scratch memory.
template <int T, int P>
void launch_tiled(const GemvArgs& p, hipStream_t st) {
  constexpr int kMost = T == FP8BQ_FP32 && P == 8 ? 3 : 5;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int nt = 1; nt <= kMost; ++nt) {
    const int64_t groups = (p.n + 16 * nt - 1) / (16 * nt) * ((p.m + 2 * P - 1) / (2 * P)), cost = (groups + 255) / 256 * (nt + 1);
    if (cost < least) least = cost, best = nt;
  }
  if (best == 1) launch_dense<T, P, 1>(p, st);
  else if (best == 2) launch_dense<T, P, 2>(p, st);
  else if (best == 3) launch_dense<T, P, 3>(p, st);
  else if constexpr (kMost == 5) {
    if (best == 4) launch_dense<T, P, 4>(p, st);
    else launch_dense<T, P, 5>(p, st);
  }
}

template <int T, int NT, int WAVES>
void launch_grouped(const GemvArgs& p, hipStream_t st) {
  const dim3 grid((unsigned)((p.n + 16 * NT - 1) / (16 * NT)), (unsigned)p.groups);
  grouped_gemv_kernel<T, NT, WAVES><<<grid, 64 * WAVES, 0, st>>>(p);
}
// Experts. Four waves share K where they all run at once (two workgroups a CU, one
// of fp32), as few rows reach few experts: a token's 8 of 32 experts, 2048 x 7168,
// 14.5 us, 18.9 with two waves. Else three tiles, for two waves where the weights
// are wide (128 rows to 32 experts of 7168 x 2048 57 us, 64 with two tiles, 71 with four
// waves) or x is fp32, for four where K gives each five chunks and there are
// enough of them (32 tokens to 32 of 256 experts, 2048 x 7168: 54 us, 61 with two
// waves; 16 rows to 16 experts at most 29, 23 with two tiles for two waves); and
// two tiles for two waves (2048 x 3584: 27 us, 29 to 32 else). The bounds are coarse:
// over 32 tokens to 32 of 256 experts, n from 1024 to 7168 and k from 2048 to 7168,
// the rule's choice is the fastest of the four or within 9% of it (three tiles for
// two waves already pay at 2560 to 3584 x 2048 or 3584, 29.0 for 31.5, and for four
// at 4096 x 5120 or 7168, 66.7 for 71.5).
// fp32, us, four waves / two: a token's 8 of 32 experts of 1024 x 2048 7.3 / 9.0, 2048 x
// 2048 11.2 / 9.7, 2048 x 7168 21.8 / 20.8; 32 tokens to 32 of 256 89 / 73.
template <int T>
void launch_experts(const GemvArgs& p, hipStream_t st) {
  constexpr bool kFp32 = T == FP8BQ_FP32;
  const int64_t tiles = (p.n + 15) / 16, reached = p.m < p.groups ? p.m : p.groups;
  if ((tiles + 1) / 2 * reached <= (kFp32 ? 256 : 512)) launch_grouped<T, 2, 4>(p, st);
  else if (kFp32 || p.n >= 4096) launch_grouped<T, 3, 2>(p, st);
  else if constexpr (!kFp32) {
    if (p.k >= 20 * 256 && (tiles + 2) / 3 * reached > 1024) launch_grouped<T, 3, 4>(p, st);
    else launch_grouped<T, 2, 2>(p, st);
  }
}

// Rows in passes of 2 P, the fewest that hold them all up to 16.
template <int T>
hipError_t run(const GemvArgs& p, hipStream_t st) {
  if (p.groups) launch_experts<T>(p, st);
  else if (p.m <= 2) launch_dense<T, 1, 1>(p, st);
  else if (p.m <= 4) launch_tiled<T, 2>(p, st);
  else if (p.m <= 8) launch_tiled<T, 4>(p, st);
  else launch_tiled<T, 8>(p, st);
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
