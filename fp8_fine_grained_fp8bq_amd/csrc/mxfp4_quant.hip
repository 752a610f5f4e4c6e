// MXFP4 quantisation (along rows, along columns, or both in one read), the
// dispatch form that picks rows by an index, and the read-back. Formats and
// layouts: include/fp8bq.h; the codec: mxfp4_codec.h. All of it is bound by
// memory: 2 (4) bytes read and 17/32 bytes written per element and form.
#include "../../include/fp8bq.h"
#include "mxfp4.h"
#include "mxfp4_codec.h"

namespace fp8bq {
namespace {

template <int T> struct Elem;
template <> struct Elem<FP8BQ_BF16> {
  using type = uint16_t;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
  static __device__ __forceinline__ uint16_t round(float v) {
    const __bf16 b = (__bf16)v;
    uint16_t r;
    __builtin_memcpy(&r, &b, 2);
    return r;
  }
};
template <> struct Elem<FP8BQ_FP16> {
  using type = uint16_t;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float value(uint16_t b) {
    _Float16 h;
    __builtin_memcpy(&h, &b, 2);
    return (float)h;
  }
  static __device__ __forceinline__ uint16_t round(float v) {
    const _Float16 h = (_Float16)v;
    uint16_t r;
    __builtin_memcpy(&r, &h, 2);
    return r;
  }
};
template <> struct Elem<FP8BQ_FP32> {
  using type = float;
  static constexpr int kBytes = 4;
  static __device__ __forceinline__ float value(float b) { return b; }
  static __device__ __forceinline__ float round(float v) { return v; }
};

// fp32 magnitude bits of the largest magnitude in the dwords w (two 16-bit
// elements each, or one fp32).
template <int T, int N>
__device__ __forceinline__ uint32_t amax_of(const uint32_t (&w)[N]) {
  uint32_t m = 0;
  if constexpr (T == FP8BQ_FP32) {
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
    return m;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) m = mx_max_pairs(m, w[i]);
    return mx_mag16<T == FP8BQ_BF16>(max(m & 0xFFFFu, m >> 16));
  }
}
// Codes of the P-th eight elements in the dwords w (the missing ones of a
// shorter w are zeros).
template <int T, int P, int N>
__device__ __forceinline__ uint32_t codes_of(const uint32_t (&w)[N], uint32_t byte) {
  if constexpr (T == FP8BQ_FP32) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 8 * P + i < N ? __uint_as_float(w[8 * P + i < N ? 8 * P + i : 0]) : 0.f;
    return mx_codes8(v, byte);
  } else {
    const uint32_t p[4] = {w[4 * P], w[4 * P + 1], w[4 * P + 2], w[4 * P + 3]};
    return mx_codes8<T == FP8BQ_BF16>(p, byte);
  }
}

// N elements of a row from column col on as dwords, zeros past `cols`. VEC: the
// row is 16-byte aligned; a group that crosses the end, and every group
// without VEC, is read element by element.
template <int T, int N, bool VEC>
__device__ __forceinline__ void load_row(const typename Elem<T>::type* row, int64_t col, int64_t cols, bool ok,
                                         uint32_t (&w)[N * Elem<T>::kBytes / 4]) {
  constexpr int kDw = N * Elem<T>::kBytes / 4;
#pragma unroll
  for (int i = 0; i < kDw; ++i) w[i] = 0;
  if (!ok || col >= cols) return;
  if (VEC && col + N <= cols) {
    const uint4* p = reinterpret_cast<const uint4*>(row + col);
#pragma unroll
    for (int i = 0; i < kDw / 4; ++i) {
      const uint4 u = p[i];
      w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (col + i < cols) {
      if constexpr (T == FP8BQ_FP32) w[i] = __float_as_uint(row[col + i]);
      else w[i / 2] |= (uint32_t)row[col + i] << (16 * (i & 1));
    }
  }
}

// The same where all of the wave's groups lie inside rows of whole 16-byte
// pieces: plain loads, which stay in flight side by side (the branches of
// load_row make the compiler wait for each before the next). The row of !ok is
// any that can be read, to be followed by clear_row.
template <int T, int N>
__device__ __forceinline__ void load_whole(const typename Elem<T>::type* row, int64_t col,
                                           uint32_t (&w)[N * Elem<T>::kBytes / 4]) {
  constexpr int kVecs = N * Elem<T>::kBytes / 16;
  const uint4* p = reinterpret_cast<const uint4*>(row + col);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const uint4 u = p[i];
    w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
  }
}
template <int N>
__device__ __forceinline__ void clear_row(bool ok, uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = ok ? w[i] : 0;
}

// DPP moves within 16-lane rows.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E;            // quad_perm [1,0,3,2], [2,3,0,1]
constexpr int kRor4 = 0x124;                         // row_ror: rotate a row of 16 lanes
constexpr int kHalfMirror = 0x141;                   // lane 7 - i of each eight
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The source row of row r of the quantised matrix; ok = false for a zero row,
// skip = true for one that the row form leaves alone.
template <bool IDX>
__device__ __forceinline__ int64_t source(const MxQuantArgs& p, int64_t r, bool& ok, bool& skip) {
  ok = r < p.rows;
  skip = !ok;
  if constexpr (IDX) {
    const int32_t t = ok ? p.src[r] : -1;
    skip = skip || t == FP8BQ_ROW_UNUSED;
    ok = t >= 0 && t < p.xrows;
    return ok ? t : 0;
  }
  return ok ? r : 0;
}

// Codes (8 bytes) and the scales' dword of the 16 elements w at place l16 of a
// 256-element chunk (16 lanes): a tile is a pair of lanes; its scale byte is
// shifted to its place in the chunk's eight, and OR over the lanes of each half
// row gives dwords, valid on lanes 4 and 12. All 16 lanes take part.
template <int T, bool NOSAT, int N>
__device__ __forceinline__ void encode_piece(const uint32_t (&w)[N], int l16, uint2& codes, uint32_t& sc) {
  uint32_t amax = amax_of<T>(w);
  amax = max2(amax, dpp<kXor1>(amax));
  const uint32_t byte = mx_scale_byte<NOSAT>(amax);
  sc = (l16 & 1) ? 0u : byte << (8 * ((l16 >> 1) & 3));
  sc |= dpp<kXor2>(sc);
  sc |= dpp<kRor4>(sc) & ((l16 & 7) < 4 ? 0u : 0xFFFFFFFFu);   // lane 4 (12) gathers lanes 0 .. 3 (8 .. 11)
  codes = make_uint2(codes_of<T, 0>(w, byte), codes_of<T, 1>(w, byte));
}
__device__ __forceinline__ void write_piece(const MxQuantArgs& p, int64_t row, int chunk, int l16, uint2 codes, uint32_t sc) {
  *reinterpret_cast<uint2*>(p.q + row * p.ldq + chunk * 128 + l16 * 8) = codes;
  if ((l16 & 7) == 4) *reinterpret_cast<uint32_t*>(p.s + ((int64_t)chunk * p.lds + row) * 8 + (l16 >> 3) * 4) = sc;
}

// Dispatch by slots: a row that several experts get is read and quantised once.
// Slot table: for each row of x the first kSlots rows that show it (in an order
// that varies from call to call and does not matter: they all get the same
// bytes) and their number. A row of zeros is written here, and so is one that
// finds its source's slots full (more than kSlots choices of a token).
constexpr int kSlots = kMxDispatchSlots;
__global__ __launch_bounds__(256) void mx_clear_kernel(int32_t* count, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) count[i] = 0;
}
template <int T, bool NOSAT, bool VEC>
__global__ __launch_bounds__(256) void mx_slot_kernel(MxQuantArgs p, int chunks, int32_t* slots, int32_t* count) {
  const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int lane = threadIdx.x & 63, l16 = lane & 15;
  const int32_t t = r < p.rows ? p.src[r] : FP8BQ_ROW_UNUSED;
  const bool real = t >= 0 && t < p.xrows;
  bool here = t != FP8BQ_ROW_UNUSED;
  if (real) {
    const int at = atomicAdd(&count[t], 1);
    here = at >= kSlots;
    if (!here) slots[(int64_t)t * kSlots + at] = (int32_t)r;
  }
  for (uint64_t left = __ballot(here); left; left &= left - 1) {   // the wave takes its lanes' rows in turn
    const int from = __ffsll((unsigned long long)left) - 1;
    const bool ok = __shfl((int)real, from) != 0;
    const int64_t row = r - lane + from, xr = ok ? __shfl(t, from) : 0;
    const auto* x = reinterpret_cast<const typename Elem<T>::type*>(p.x) + xr * p.ldx;
    for (int c0 = 0; c0 < chunks; c0 += 4) {
      const int chunk = c0 + (lane >> 4);
      uint32_t w[16 * Elem<T>::kBytes / 4], sc;
      load_row<T, 16, VEC>(x, (int64_t)chunk * 256 + l16 * 16, p.cols, ok, w);
      uint2 codes;
      encode_piece<T, NOSAT>(w, l16, codes, sc);
      if (chunk < chunks) write_piece(p, row, chunk, l16, codes, sc);
    }
  }
}

// Row form. 16 lanes take one 256-element chunk of a row, 16 elements each (32
// contiguous bytes of bf16), so a lane's codes are one 8-byte store; each lane
// takes the same place of two neighbouring chunks, all loads before any
// arithmetic. A block takes 16 rows of a chunk pair, the pairs of a row run
// fastest over the grid. 16384 x 7168 bf16: 44 us, 6.7 TB/s. SLOTS: rows of x, each written to the rows in its slots.
template <int T, bool NOSAT, bool IDX, bool VEC, bool SLOTS = false>
__global__ __launch_bounds__(256) void mx_quant_rows_kernel(MxQuantArgs p, int chunks, const int32_t* slots = nullptr,
                                                            const int32_t* count = nullptr) {
  const int t = threadIdx.x, l16 = t & 15;
  const unsigned pairs = (unsigned)(chunks + 1) / 2;
  const int chunk0 = 2 * (int)(blockIdx.x % pairs);
  const int64_t r = (int64_t)(blockIdx.x / pairs) * 16 + (t >> 4);
  bool ok, skip;
  int64_t xr;
  int n = 1;
  if constexpr (SLOTS) {
    n = r < p.xrows ? min(count[r], kSlots) : 0;
    ok = n > 0;                                         // a row that nobody gets is not read
    skip = !ok;
    xr = ok ? r : 0;
  } else {
    xr = source<IDX>(p, r, ok, skip);
  }
  if (skip) return;                                     // all 16 lanes of the row
  uint32_t w[2][16 * Elem<T>::kBytes / 4];
  const auto* row = reinterpret_cast<const typename Elem<T>::type*>(p.x) + xr * p.ldx;
  if (VEC && ((int64_t)chunk0 + 2) * 256 <= p.cols) {   // uniform
#pragma unroll
    for (int u = 0; u < 2; ++u) load_whole<T, 16>(row, (int64_t)(chunk0 + u) * 256 + l16 * 16, w[u]);
#pragma unroll
    for (int u = 0; u < 2; ++u) clear_row(ok, w[u]);
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u) load_row<T, 16, VEC>(row, (int64_t)(chunk0 + u) * 256 + l16 * 16, p.cols, ok, w[u]);
  }
  int32_t to[SLOTS ? kSlots : 1];
  if constexpr (SLOTS) {
    static_assert(kSlots % 4 == 0, "slots are read four at a time");
#pragma unroll
    for (int i = 0; i < kSlots / 4; ++i)
      *reinterpret_cast<int4*>(&to[4 * i]) = reinterpret_cast<const int4*>(slots + xr * kSlots)[i];
  }
  uint2 codes[2];
  uint32_t sc[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) encode_piece<T, NOSAT>(w[u], l16, codes[u], sc[u]);
#pragma unroll
  for (int i = 0; i < (SLOTS ? kSlots : 1); ++i) {
    if (i >= n) break;
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (chunk0 + u < chunks) write_piece(p, SLOTS ? to[i] : r, chunk0 + u, l16, codes[u], sc[u]);
  }
}

// Column form, and (ROWS) the row form beside it from the same read. A block
// stages 128 rows of 128 bytes (64 columns, 32 of fp32) in LDS; then thread
// (column dword, row tile, half of the dword) walks 32 rows of its dword:
// consecutive lanes on consecutive dwords, 16 bytes of codes per thread. The
// four row tiles' scale bytes of a column meet in LDS for one 4-byte store. The
// grid covers whole 256 x 256 squares of the matrix (what lies past it is
// zeros); the blocks of a square run on one XCD, one after the other, so that
// the pieces of code rows that they write (32 bytes of a row, 64 of a column)
// meet as full lines in its L2. The squares run over the columns first. Bound
// by its phases (a block reads, then computes, then writes) with eight blocks on
// a CU: both forms of 16384 x 7168 bf16 in 72 us (5.0 TB/s; the row form alone 44,
// 6.7), of 4096 x 7168 in 18. Persistent blocks that read the next tile during
// this one's columns: 90 and 17.6; 128 x 128 tiles: 4.2 TB/s.
constexpr int kColsThreads = 256;
template <int T, bool NOSAT, bool IDX, bool VEC, bool ROWS>
__global__ __launch_bounds__(kColsThreads) void mx_quant_cols_kernel(MxQuantArgs p, unsigned rsq, unsigned csq) {
  constexpr int kPer = 4 / Elem<T>::kBytes;             // elements per dword
  constexpr int kCols = 32 * kPer;
  constexpr int kLane = 4 * kPer;                       // elements of a lane's 16 bytes
  constexpr int kRounds = 128 * 8 / kColsThreads;       // rows per thread of the load
  constexpr int kStep = kColsThreads / 8;
  __shared__ uint32_t tile[128][32];
  __shared__ uint8_t scales[kCols][4];
  const int t = threadIdx.x, l8 = t & 7;
  constexpr int kSub = 2 * 256 / kCols;                 // blocks of a square
  const unsigned g = blockIdx.x / (8 * kSub), in = blockIdx.x % (8 * kSub);
  const unsigned here = min(rsq * csq - 8 * g, 8u);     // squares of this group of (up to) eight, one per XCD
  const unsigned sq = 8 * g + in % here, sub = in / here;
  const int64_t r0 = (int64_t)(sq / csq) * 256 + (sub & 1) * 128, c0 = (int64_t)(sq % csq) * 256 + (sub >> 1) * kCols;

  uint32_t w[kRounds][4];
  bool ok[kRounds], skip[kRounds];
  const typename Elem<T>::type* row[kRounds];
#pragma unroll
  for (int i = 0; i < kRounds; ++i)
    row[i] = reinterpret_cast<const typename Elem<T>::type*>(p.x) +
             source<IDX>(p, r0 + i * kStep + (t >> 3), ok[i], skip[i]) * p.ldx;
  if (VEC && c0 + kCols <= p.cols) {                    // uniform
#pragma unroll
    for (int i = 0; i < kRounds; ++i) load_whole<T, kLane>(row[i], c0 + l8 * kLane, w[i]);
#pragma unroll
    for (int i = 0; i < kRounds; ++i) clear_row(ok[i], w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kRounds; ++i) load_row<T, kLane, VEC>(row[i], c0 + l8 * kLane, p.cols, ok[i], w[i]);
  }
#pragma unroll
  for (int i = 0; i < kRounds; ++i)
    *reinterpret_cast<uint4*>(&tile[i * kStep + (t >> 3)][l8 * 4]) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);

  if constexpr (ROWS) {
    // a tile is 4 lanes (8 of fp32); its scale byte sits on all of them
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int64_t r = r0 + i * kStep + (t >> 3);
      uint32_t amax = amax_of<T>(w[i]);
      amax = max2(amax, dpp<kXor1>(amax));
      amax = max2(amax, dpp<kXor2>(amax));
      if constexpr (kPer == 1) amax = max2(amax, dpp<kHalfMirror>(amax));
      const uint32_t byte = mx_scale_byte<NOSAT>(amax);
      const uint32_t code = codes_of<T, 0>(w[i], byte);
      uint8_t* sp = p.s + ((c0 / 256) * p.lds + r) * 8 + (c0 % 256) / 32;
      if constexpr (kPer == 2) {
        uint32_t sc = byte << (8 * (l8 >> 2));
        sc |= dpp<kHalfMirror>(sc);
        if (!skip[i]) {
          *reinterpret_cast<uint32_t*>(p.q + r * p.ldq + c0 / 2 + l8 * 4) = code;
          if (l8 == 0) *reinterpret_cast<uint16_t*>(sp) = (uint16_t)sc;
        }
      } else if (!skip[i]) {
        *reinterpret_cast<uint16_t*>(p.q + r * p.ldq + c0 / 2 + l8 * 2) = (uint16_t)code;
        if (l8 == 0) *sp = (uint8_t)byte;
      }
    }
  }
  __syncthreads();

  const int cd = t & 31, rt = (t >> 5) & 3, h = t >> 7;
  if (h < kPer) {
    uint32_t d[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) d[i] = tile[rt * 32 + i][cd];
    // the 32 rows of this dword's h-th column: fp32 as they are, 16-bit ones regrouped two rows to a dword
    constexpr int kDw = 32 / kPer;
    const uint32_t pick = h ? 0x07060302u : 0x05040100u;
    uint32_t v[kDw];
#pragma unroll
    for (int i = 0; i < kDw; ++i) {
      if constexpr (kPer == 1) v[i] = d[i];
      else v[i] = __builtin_amdgcn_perm(d[2 * i + 1], d[2 * i], pick);
    }
    const uint32_t byte = mx_scale_byte<NOSAT>(amax_of<T>(v));
    scales[cd * kPer + h][rt] = (uint8_t)byte;
    const int64_t c = c0 + cd * kPer + h;
    if (c < p.cols)
      *reinterpret_cast<uint4*>(p.qt + c * p.ldqt + r0 / 2 + rt * 16) =
          make_uint4(codes_of<T, 0>(v, byte), codes_of<T, 1>(v, byte), codes_of<T, 2>(v, byte), codes_of<T, 3>(v, byte));
  }
  __syncthreads();
  if (t < kCols && c0 + t < p.cols)
    *reinterpret_cast<uint32_t*>(p.st + ((r0 / 256) * p.ldst + c0 + t) * 8 + (r0 % 256) / 32) =
        *reinterpret_cast<const uint32_t*>(scales[t]);
}

// Read-back: 32 lanes take a chunk of a row, 8 codes each, so that a wave's
// stores of bf16 are contiguous; four rows per thread, all loads first.
template <int T, bool VEC>
__global__ __launch_bounds__(256) void mx_dequant_kernel(const uint8_t* __restrict__ q, int64_t rows, int64_t cols,
                                                         int64_t ldq, const uint8_t* __restrict__ s, int64_t lds,
                                                         typename Elem<T>::type* __restrict__ y, int64_t ldy,
                                                         int chunks) {
  const int t = threadIdx.x, l32 = t & 31;
  const int chunk = (int)(blockIdx.x % (unsigned)chunks);
  const int64_t r0 = (int64_t)(blockIdx.x / (unsigned)chunks) * 32 + (t >> 5);
  const int64_t c = (int64_t)chunk * 256 + l32 * 8;
  if (c >= cols) return;
  uint32_t codes[4], byte[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t r = min(r0 + 8 * u, rows - 1);
    codes[u] = *reinterpret_cast<const uint32_t*>(q + r * ldq + chunk * 128 + l32 * 4);
    byte[u] = s[((int64_t)chunk * lds + r) * 8 + (l32 >> 2)];
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t r = r0 + 8 * u;
    if (r >= rows) return;
    const float sc = mx_scale(byte[u]);
    typename Elem<T>::type o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t code = (codes[u] >> (4 * i)) & 15u;
      // E2M1 to fp32: exponent field 0 holds 0 and 0.5, else (1 + m / 2) * 2^(e - 1)
      const uint32_t em = code & 7u;
      const uint32_t mag = em >= 2 ? (em << 22) + (126u << 23) : (em ? 126u << 23 : 0u);
      o[i] = Elem<T>::round(__uint_as_float(mag | ((code & 8u) << 28)) * sc);
    }
    auto* dst = y + r * ldy + c;
    if (VEC && c + 8 <= cols) {
      constexpr int kVecs = 8 * Elem<T>::kBytes / 16;
      uint4 v[kVecs];
      __builtin_memcpy(v, o, sizeof(v));
#pragma unroll
      for (int i = 0; i < kVecs; ++i) reinterpret_cast<uint4*>(dst)[i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < cols) dst[i] = o[i];
    }
  }
}

template <int T, bool NOSAT, bool IDX, bool VEC>
hipError_t run_quant(const MxQuantArgs& a, int32_t* ws, hipStream_t st) {
  const int cchunks = (int)((a.cols + 255) / 256);
  if (a.qt) {
    constexpr int kCols = 32 * 4 / Elem<T>::kBytes;
    const unsigned rsq = (unsigned)((a.rows + 255) / 256);
    const unsigned grid = rsq * (unsigned)cchunks * (2 * 256 / kCols);
    if (a.q) mx_quant_cols_kernel<T, NOSAT, IDX, VEC, true><<<grid, kColsThreads, 0, st>>>(a, rsq, cchunks);
    else mx_quant_cols_kernel<T, NOSAT, IDX, VEC, false><<<grid, kColsThreads, 0, st>>>(a, rsq, cchunks);
  } else if (IDX && ws) {
    int32_t *slots = ws, *count = ws + a.xrows * kSlots;
    mx_clear_kernel<<<(unsigned)((a.xrows + 255) / 256), 256, 0, st>>>(count, a.xrows);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    mx_slot_kernel<T, NOSAT, VEC><<<(unsigned)((a.rows + 255) / 256), 256, 0, st>>>(a, cchunks, slots, count);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const unsigned blocks = (unsigned)((a.xrows + 15) / 16) * (unsigned)((cchunks + 1) / 2);
    mx_quant_rows_kernel<T, NOSAT, IDX, VEC, true><<<blocks, 256, 0, st>>>(a, cchunks, slots, count);
  } else {
    const unsigned blocks = (unsigned)((a.rows + 15) / 16) * (unsigned)((cchunks + 1) / 2);
    mx_quant_rows_kernel<T, NOSAT, IDX, VEC><<<blocks, 256, 0, st>>>(a, cchunks);
  }
  return hipGetLastError();
}

template <int T>
hipError_t pick_quant(const MxQuantArgs& a, bool nosat, int32_t* ws, hipStream_t st) {
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx * Elem<T>::kBytes % 16 == 0;
  const int sel = (nosat ? 4 : 0) + (a.src ? 2 : 0) + (vec ? 1 : 0);
  switch (sel) {
    case 0: return run_quant<T, false, false, false>(a, ws, st);
    case 1: return run_quant<T, false, false, true>(a, ws, st);
    case 2: return run_quant<T, false, true, false>(a, ws, st);
    case 3: return run_quant<T, false, true, true>(a, ws, st);
    case 4: return run_quant<T, true, false, false>(a, ws, st);
    case 5: return run_quant<T, true, false, true>(a, ws, st);
    case 6: return run_quant<T, true, true, false>(a, ws, st);
    default: return run_quant<T, true, true, true>(a, ws, st);
  }
}

template <int T>
hipError_t run_dequant(const uint8_t* q, int64_t rows, int64_t cols, int64_t ldq, const uint8_t* s, int64_t lds,
                       void* y, int64_t ldy, hipStream_t st) {
  using E = typename Elem<T>::type;
  const int chunks = (int)((cols + 255) / 256);
  const unsigned blocks = (unsigned)((rows + 31) / 32) * (unsigned)chunks;
  E* out = static_cast<E*>(y);
  if (reinterpret_cast<uintptr_t>(y) % 16 == 0 && ldy * Elem<T>::kBytes % 16 == 0)
    mx_dequant_kernel<T, true><<<blocks, 256, 0, st>>>(q, rows, cols, ldq, s, lds, out, ldy, chunks);
  else
    mx_dequant_kernel<T, false><<<blocks, 256, 0, st>>>(q, rows, cols, ldq, s, lds, out, ldy, chunks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_mxfp4(const MxQuantArgs& a, int xtype, bool nosat, int32_t* ws, hipStream_t stream) {
  switch (xtype) {
    case FP8BQ_BF16: return pick_quant<FP8BQ_BF16>(a, nosat, ws, stream);
    case FP8BQ_FP16: return pick_quant<FP8BQ_FP16>(a, nosat, ws, stream);
    default: return pick_quant<FP8BQ_FP32>(a, nosat, ws, stream);
  }
}

hipError_t launch_dequant_mxfp4(const uint8_t* q, int64_t rows, int64_t cols, int64_t ldq, const uint8_t* s,
                                int64_t lds, void* y, int ytype, int64_t ldy, hipStream_t stream) {
  switch (ytype) {
    case FP8BQ_BF16: return run_dequant<FP8BQ_BF16>(q, rows, cols, ldq, s, lds, y, ldy, stream);
    case FP8BQ_FP16: return run_dequant<FP8BQ_FP16>(q, rows, cols, ldq, s, lds, y, ldy, stream);
    default: return run_dequant<FP8BQ_FP32>(q, rows, cols, ldq, s, lds, y, ldy, stream);
  }
}

}  // namespace fp8bq
