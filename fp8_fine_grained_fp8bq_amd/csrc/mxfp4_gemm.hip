// MXFP4 products out = A B^T for gfx950: dense, over rows grouped by expert, and
// over the K axis grouped by expert (weight gradients). Formats and layouts:
// include/fp8bq.h.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 on E2M1 operands: lane l holds row l % 32 of
// each operand and the 32 codes (16 bytes) of K-block l / 32, with that block's
// E8M0 byte picked from a dword by op_sel. Any order of K-blocks that both
// operands share gives the same sum, so lane half h takes blocks 4 h .. 4 h + 3
// of a 256-element chunk in four MFMAs: its codes are 64 contiguous bytes of
// the row and its four scale bytes one dword. The weight side (B) is the
// first operand: lane l's sixteen results are row l % 32 of A and, register r,
// column 8 (r / 4) + 4 (l / 32) + r % 4 of B.
#include <utility>

#include "gemm_kernels.h"
#include "mxfp4.h"

namespace fp8bq {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  const __bf16 b = (__bf16)v;
  uint16_t r;
  __builtin_memcpy(&r, &b, 2);
  return r;
}

// acc += over the two K-blocks of MFMA t (0 .. 3) of a chunk.
template <int T>
__device__ __forceinline__ v16f mfma(const uint4& b, const uint4& a, const v16f& acc, int sb, int sa) {
  const v8i x = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  const v8i y = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc, 4, 4, T, sb, T, sa);
}

// Bounds of group e in a device table of offsets: clamped into [0, limit], and
// not below its start.
__device__ __forceinline__ void group_range(const int32_t* off, int e, int64_t limit, int64_t& lo, int64_t& hi) {
  lo = min(max((int64_t)off[e], (int64_t)0), limit);
  hi = min(max((int64_t)off[e + 1], lo), limit);
}

// Row tile `tile` of height H over the groups' rows, each group's tiles
// counted up from its first row: the group and the rows, or e = -1 past the
// last. A wave looks at four groups per lane (at most 256 in all).
struct RowTile { int e; int64_t m0, m_end; };
template <int H>
__device__ __forceinline__ RowTile find_tile(const int32_t* off, int groups, int64_t limit, int tile) {
  const int lane = threadIdx.x & 63;
  int64_t lo[4], hi[4];
  int cnt[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane * 4 + i;
    lo[i] = hi[i] = 0;
    if (e < groups) group_range(off, e, limit, lo[i], hi[i]);
    cnt[i] = (int)((hi[i] - lo[i] + H - 1) / H);
    sum += cnt[i];
  }
  int before = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(before, d);
    if (lane >= d) before += v;
  }
  before -= sum;                                   // tiles before this lane's groups
  int e = -1, m0 = 0, m_end = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (tile >= before && tile < before + cnt[i]) {
      e = lane * 4 + i;
      m0 = (int)lo[i] + (tile - before) * H;
      m_end = min(m0 + H, (int)hi[i]);
    }
    before += cnt[i];
  }
  const uint64_t hit = __ballot(e >= 0);
  if (hit == 0) return {-1, 0, 0};
  const int from = __ffsll((unsigned long long)hit) - 1;
  return {__builtin_amdgcn_readfirstlane(__shfl(e, from)), __builtin_amdgcn_readfirstlane(__shfl(m0, from)),
          __builtin_amdgcn_readfirstlane(__shfl(m_end, from))};
}

// One 32 x 32 output tile per workgroup; its WAVES waves take the chunks of K
// in turn, straight from memory into registers, and meet in LDS at the end
// (added in the order of waves).
template <int MODE, bool F32, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void mx_stream_kernel(MxGemmArgs p) {
  __shared__ float part[WAVES][16][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;

  const unsigned tiles_n = (unsigned)((p.n + 31) / 32);
  const int tm = (int)(blockIdx.x / tiles_n);
  const int64_t n0 = (int64_t)(blockIdx.x % tiles_n) * 32;
  int64_t m0 = (int64_t)tm * 32, m_end = min(m0 + 32, p.m);
  const uint8_t* b = p.b;
  const uint8_t* sb = p.sb;
  int64_t out_base = 0;
  int c0 = 0, c1 = p.chunks;
  if constexpr (MODE == MX_ROWS) {
    const RowTile t = find_tile<32>(p.row_off, p.groups, p.m, tm);
    if (t.e < 0) return;
    m0 = t.m0;
    m_end = t.m_end;
    b += (int64_t)t.e * p.n * p.ldb;
    sb += (int64_t)t.e * p.chunks * p.ldsb * 8;
  }
  if constexpr (MODE == MX_K) {
    const int e = blockIdx.y;
    int64_t lo, hi;
    group_range(p.row_off, e, (int64_t)p.chunks * 256, lo, hi);
    c0 = (int)(lo / 256);
    c1 = (int)(hi / 256);
    out_base = (int64_t)e * p.m * p.ldo;
  }

  // rows past the end repeat the last one (their results are not stored)
  const int64_t ra = min(m0 + r, m_end - 1), rb = min(n0 + r, p.n - 1);
  const uint8_t* pa = p.a + ra * p.lda + h * 64;
  const uint8_t* pb = b + rb * p.ldb + h * 64;
  const uint8_t* psa = p.sa + ra * 8 + h * 4;
  const uint8_t* psb = sb + rb * 8 + h * 4;

  v16f acc;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  // two chunks' loads in flight per wave
  struct Chunk { uint4 a[4], b[4]; int ea, eb; };
  auto load = [&](Chunk& k, int c) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      k.b[t] = *reinterpret_cast<const uint4*>(pb + (int64_t)c * 128 + t * 16);
      k.a[t] = *reinterpret_cast<const uint4*>(pa + (int64_t)c * 128 + t * 16);
    }
    k.ea = *reinterpret_cast<const int*>(psa + (int64_t)c * p.ldsa * 8);
    k.eb = *reinterpret_cast<const int*>(psb + (int64_t)c * p.ldsb * 8);
  };
  auto use = [&](const Chunk& k) {
    acc = mfma<0>(k.b[0], k.a[0], acc, k.eb, k.ea);
    acc = mfma<1>(k.b[1], k.a[1], acc, k.eb, k.ea);
    acc = mfma<2>(k.b[2], k.a[2], acc, k.eb, k.ea);
    acc = mfma<3>(k.b[3], k.a[3], acc, k.eb, k.ea);
  };
  for (int c = c0 + wave; c < c1; c += 2 * WAVES) {
    Chunk x, y;
    load(x, c);
    if (c + WAVES < c1) {                          // uniform
      load(y, c + WAVES);
      use(x);
      use(y);
    } else {
      use(x);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  for (int u = tid; u < 1024; u += 64 * WAVES) {
    const int reg = u >> 6, l = u & 63;
    float v = part[0][reg][l];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += part[w][reg][l];
    const int64_t row = m0 + (l & 31), col = n0 + 8 * (reg >> 2) + 4 * (l >> 5) + (reg & 3);
    if (row < m_end && col < p.n) {
      if constexpr (F32) static_cast<float*>(p.out)[out_base + row * p.ldo + col] = v;
      else static_cast<uint16_t*>(p.out)[out_base + row * p.ldo + col] = bf16_bits(v);
    }
  }
}

// ---------------------------------------------------------------------------
// Tiled kernel. Workgroup tile 64 TM x 64 TN, four waves (one per SIMD) of
// 32 TM x 32 TN; a step is one 256-element chunk: 128 bytes of each operand row
// and 8 scale bytes. Persistent workgroups walk the output tiles; operands go
// global -> LDS by LDS DMA two steps ahead into two stages (the FP8 kernels'
// loads, swizzle and tile walk; an E2M1 chunk has the bytes of an FP8 one and
// twice the products).
//
// A step is four slices of TM x TN MFMAs (slice t: K-blocks t and 4 + t of the
// chunk). Each slice has its own fragment registers: while slice t runs, the
// fragments that slice t - 1 used are read for the step they are needed in
// next, so that every LDS read has a slice or more to land:
//   slice 0: reads slice 3 of this step, then the one barrier of the step
//            (every wave has read all of this stage, the other one has landed);
//   slices 1 .. 3: read slices 0 .. 2 of the next step, and send the loads of
//            NST steps on into this step's stage, spread evenly.
// Eight waves of half the tile each (two per SIMD, half the accumulators) took
// the same time: the step of 64 MFMAs (2048 cycles) takes 2280 without its 68
// loads of 1 KB and 2630 .. 2700 with them, whichever way they are spread, at a
// clock of 1.6 .. 1.7 GHz that the power budget sets (with all-zero codes the
// same kernel runs 25% faster; MFMAs alone on random codes reach 6.8 of the
// nominal 9.9 PFLOP/s at 1.7 GHz).
// SPLIT: four waves compute and four more only load. A 1 KB load holds its wave
// up for 64 .. 90 cycles when four waves load at once (the CU takes in about 64
// bytes a cycle), two or three MFMAs' time; where a tile's step has few MFMAs to
// hide that behind (48 x 18432 x 7168 in tiles of 64 x 128: 14.9 against 17.2 us
// without; 8 experts' 822 rows: 21.0 against 22.1), and there are too few tiles
// for a second workgroup on the CU to fill the gaps, the loads get their own
// waves. The large tiles leave no registers for that.
// The accumulators sit in the AGPRs (256 of them at TM = TN = 4), tied to the
// MFMA statements as in the power-of-two FP8 kernel.
// ---------------------------------------------------------------------------
typedef int v4i __attribute__((ext_vector_type(4)));

template <int TM, int TN>
struct TileCfg {
  static constexpr int kBM = 64 * TM, kBN = 64 * TN;
  static constexpr int kBOff = kBM * 128;
  static constexpr int kSaOff = (kBM + kBN) * 128;
  static constexpr int kSbOff = kSaOff + (kBM < 128 ? 128 : kBM) * 8;   // a scale load covers 128 rows
  static constexpr int kStage = kSbOff + (kBN < 128 ? 128 : kBN) * 8;
  static constexpr int kRoundsA = kBM / 32, kRoundsB = kBN / 32;        // loads per wave: 8 rows each
  static constexpr int kParts = kRoundsA + kRoundsB + 1;
};

// acc += over slice T. The compiler does not see the instruction's hazards: an
// operand that a VALU instruction has just written needs two wait states.
// Fragments come from LDS reads (waited for by the compiler); the exponents
// and the cleared accumulators come from VALU moves, which exponents_ready()
// follows. WAIT: the two states before every MFMA, for the small tiles, whose
// registers the compiler may park in AGPRs and fetch back right before use; for
// the large ones they would cost 2 .. 3% (987 against 970 us on 16384 x 18432 x
// 7168). tests/test_mfma_hazards.py checks the built code of both.
// One statement each, so that nothing comes between the wait and the MFMA.
#define FP8BQ_MFMA(wait, sel) \
  asm volatile(wait "v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 " sel " cbsz:4 blgp:4" \
               : "+a"(acc) : "v"(b), "v"(a), "v"(sb), "v"(sa))
#define FP8BQ_MFMA_SLICE(wait) \
  if constexpr (T == 0) FP8BQ_MFMA(wait, "op_sel_hi:[0,0,0]"); \
  else if constexpr (T == 1) FP8BQ_MFMA(wait, "op_sel:[1,1,0] op_sel_hi:[0,0,0]"); \
  else if constexpr (T == 2) FP8BQ_MFMA(wait, "op_sel_hi:[1,1,0]"); \
  else FP8BQ_MFMA(wait, "op_sel:[1,1,0] op_sel_hi:[1,1,0]")
template <int T, bool WAIT>
__device__ __forceinline__ void mfma_slice(v16f& acc, const v4i& b, const v4i& a, int sb, int sa) {
  if constexpr (WAIT) {
    FP8BQ_MFMA_SLICE("s_nop 1\n\t");
  } else {
    FP8BQ_MFMA_SLICE("");
  }
}
#undef FP8BQ_MFMA_SLICE
#undef FP8BQ_MFMA
__device__ __forceinline__ void exponents_ready() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 3" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Waits until at most N of the wave's vector memory operations are left.
template <int N>
__device__ __forceinline__ void wait_loads_left() {
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}

struct MxTile {
  int64_t m0, m_end, n0;
  int e, c0, nc;                 // group, first chunk, chunks
};

// Group tables in LDS (rows or chunks of each group; row tiles before it).
struct MxTables {
  int lo[256], hi[256], before[257];
};

template <int MODE, int TM, int TN>
struct MxWalk {
  using C = TileCfg<TM, TN>;
  const MxGemmArgs& p;
  const MxTables& tab;
  int tiles_m, tiles_n, total, start, nper, mine;

  // Workgroup w runs on XCD w % 8. A grid of 8 C workgroups deals chunks of C
  // consecutive tiles to the XCDs in turn, so that an XCD's workgroups share
  // operand panels in its L2 at any time; another grid (fewer tiles than CUs)
  // gives XCD x a contiguous range.
  __device__ __forceinline__ MxWalk(const MxGemmArgs& p_, const MxTables& tab_) : p(p_), tab(tab_) {
    tiles_n = (int)((p.n + C::kBN - 1) / C::kBN);
    tiles_m = MODE == MX_ROWS ? tab.before[p.groups] : (int)((p.m + C::kBM - 1) / C::kBM);
    total = tiles_m * tiles_n * (MODE == MX_K ? p.groups : 1);
    const int G = gridDim.x, w = blockIdx.x, x = w % kXcds, local = w / kXcds;
    if (G % kXcds == 0) {
      start = x * (G / kXcds) + local;
      nper = G;
      mine = start < total ? (total - 1 - start) / G + 1 : 0;
    } else {
      nper = G / kXcds + (x < G % kXcds ? 1 : 0);
      const int count = total / kXcds + (x < total % kXcds ? 1 : 0);
      start = x * (total / kXcds) + min(x, total % kXcds) + local;
      mine = local < count ? (count - local + nper - 1) / nper : 0;
    }
    total = __builtin_amdgcn_readfirstlane(total);
    mine = __builtin_amdgcn_readfirstlane(mine);
  }

  // This workgroup's t-th tile: row tiles in groups of 8, columns within.
  __device__ __forceinline__ MxTile tile(int t) const {
    int logical = start + nper * t;
    MxTile r;
    r.e = 0;
    r.c0 = 0;
    r.nc = p.chunks;
    if constexpr (MODE == MX_K) {
      r.e = logical / (tiles_m * tiles_n);
      logical -= r.e * tiles_m * tiles_n;
      r.c0 = __builtin_amdgcn_readfirstlane(tab.lo[r.e]);
      r.nc = __builtin_amdgcn_readfirstlane(tab.hi[r.e]) - r.c0;
    }
    const int per = kGroupM * tiles_n, group = logical / per, first = group * kGroupM;
    const int size = min(tiles_m - first, kGroupM), in = logical - group * per;
    const int tm = first + in % size, tn = in / size;
    if constexpr (MODE == MX_ROWS) {
      int lo = 0, hi = p.groups;                 // e: before[e] <= tm < before[e + 1]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__builtin_amdgcn_readfirstlane(tab.before[mid]) <= tm) lo = mid; else hi = mid;
      }
      r.e = lo;
      r.m0 = __builtin_amdgcn_readfirstlane(tab.lo[lo]) + (int64_t)(tm - __builtin_amdgcn_readfirstlane(tab.before[lo])) * C::kBM;
      r.m_end = min(r.m0 + C::kBM, (int64_t)__builtin_amdgcn_readfirstlane(tab.hi[lo]));
    } else {
      r.m0 = (int64_t)tm * C::kBM;
      r.m_end = min(r.m0 + C::kBM, p.m);
    }
    r.n0 = (int64_t)tn * C::kBN;
    return r;
  }
};

// The loads: wave w brings rows 32 i + 8 w .. + 7 of either operand in round i
// (lane l: row l / 8 of them, 16 bytes at physical slot l % 8, that is logical
// slot (l % 8) ^ swz(row)), and 128 rows' scales: waves 0 and 1 of A, 2 and 3
// of B. Raw buffer resources end with the operand: what lies past it reads as
// zeros, dword by dword. After the last step the cursor stays where it is and
// the loads repeat into a stage that nobody reads.
template <int MODE, int TM, int TN>
struct MxLoader {
  using C = TileCfg<TM, TN>;
  const MxGemmArgs& p;
  const MxWalk<MODE, TM, TN>& wk;
  const uint32_t smem;
  const int wave;
  uint32_t voff_a[C::kRoundsA], voff_b[C::kRoundsB], voff_s;
  u32x4 rs_a, rs_b, rs_s;
  const uint8_t *s_at, *s_end;           // the scales' resource spans a whole array, which may exceed its 4 GiB
  int tk = 0, c = 0, nc = 0;

  __device__ __forceinline__ MxLoader(const MxGemmArgs& p_, const MxWalk<MODE, TM, TN>& wk_, uint32_t smem_, int wave_,
                                      int lane)
      : p(p_), wk(wk_), smem(smem_), wave(wave_) {
    const uint32_t row = 8 * wave + (lane >> 3);
    const uint32_t g16 = (uint32_t)(((lane & 7) ^ (lane >> 3) ^ (wave & 1)) * 16);
#pragma unroll
    for (int i = 0; i < C::kRoundsA; ++i) voff_a[i] = (32 * i + row) * (uint32_t)p.lda + g16;
#pragma unroll
    for (int i = 0; i < C::kRoundsB; ++i) voff_b[i] = (32 * i + row) * (uint32_t)p.ldb + g16;
    voff_s = (uint32_t)((wave & 1) * 128 + 2 * lane) * 8;
    while (tk < wk.mine && wk.tile(tk).nc == 0) ++tk;      // K groups without rows
    open();
  }
  __device__ __forceinline__ void open() {
    if (tk >= wk.mine) tk = 0;                             // nothing to load at all: nobody reads the stage
    const MxTile t = wk.tile(tk);
    nc = t.nc;
    c = 0;
    const uint8_t* b = p.b;
    const uint8_t* sb = p.sb;
    if constexpr (MODE == MX_ROWS) {
      b += (int64_t)t.e * p.n * p.ldb;
      sb += (int64_t)t.e * p.chunks * p.ldsb * 8;
    }
    const int64_t k0 = (int64_t)t.c0 * 128;
    rs_a = make_rsrc(p.a + t.m0 * p.lda + k0, p.a + (p.m - 1) * p.lda + (int64_t)p.chunks * 128);
    rs_b = make_rsrc(b + t.n0 * p.ldb + k0, b + (p.n - 1) * p.ldb + (int64_t)p.chunks * 128);
    if (wave < 2) {
      s_at = p.sa + ((int64_t)t.c0 * p.ldsa + t.m0) * 8;
      s_end = p.sa + ((int64_t)(p.chunks - 1) * p.ldsa + p.m) * 8;
    } else {
      s_at = sb + ((int64_t)t.c0 * p.ldsb + t.n0) * 8;
      s_end = sb + ((int64_t)(p.chunks - 1) * p.ldsb + p.n) * 8;
    }
    rs_s = make_rsrc(s_at, s_end);
  }
  __device__ __forceinline__ void advance() {
    if (c + 1 < nc) {
      ++c;
      bump_rsrc(rs_a, 128);
      bump_rsrc(rs_b, 128);
      s_at += (wave < 2 ? p.ldsa : p.ldsb) * 8;
      rs_s = make_rsrc(s_at, s_end);
      return;
    }
    int next = tk + 1;
    if constexpr (MODE == MX_K) while (next < wk.mine && wk.tile(next).nc == 0) ++next;
    if (next < wk.mine) {
      tk = next;
      open();
    }
  }
  __device__ __forceinline__ void part(int q, int stage) const {
    const uint32_t base = smem + (uint32_t)(stage * C::kStage);
    if (q < C::kRoundsA) dma16_buf(rs_a, voff_a[q], base + (32 * q + 8 * wave) * 128);
    else if (q < C::kRoundsA + C::kRoundsB)
      dma16_buf(rs_b, voff_b[q - C::kRoundsA], base + C::kBOff + (32 * (q - C::kRoundsA) + 8 * wave) * 128);
    else if (brings_scales())
      dma16_buf(rs_s, voff_s, base + (wave < 2 ? C::kSaOff : C::kSbOff) + (wave & 1) * 1024);
  }
  __device__ __forceinline__ bool brings_scales() const { return (wave & 1) * 128 < (wave < 2 ? C::kBM : C::kBN); }
};

// ---- epilogue ------------------------------------------------------------------
// Lanes hold columns 8 q + 4 h .. + 3 (q = 0 .. 3, h = l / 32) of row l % 32; the
// stores write whole 128-byte lines, 8 rows to an instruction. Four lanes are
// brought onto one row by row swaps (v_permlane32_swap, v_permlane16_swap), and
// eight by a rotation within 16-lane rows.

// 16 bytes per lane. Whole lines are stored past the caches (LINE), measured
// against plain stores in turn on one card: 54066 rows of 8 experts, n = 2048, k =
// 7168: 367 against 383 us; 32 fp32 gradients of 1024 x 2048: 59 against 91 (with
// half lines 84); 4096 x 7168 x 2048: 40.5 against 41.7 (with half lines 45.9). On
// other cards, and behind a step's other kernels, the first are 370 .. 485, 64 ..
// 68 and 42.
typedef uint32_t u32x4s __attribute__((ext_vector_type(4)));
template <bool LINE>
__device__ __forceinline__ void put16(void* p, const uint32_t (&v)[4]) {
  const u32x4s w = {v[0], v[1], v[2], v[3]};
  if constexpr (LINE) __builtin_nontemporal_store(w, static_cast<u32x4s*>(p));
  else *static_cast<u32x4s*>(p) = w;
}

// x and y: 16 bytes each of rows l % 16 (64-byte halves of their lines, x the
// first). Becomes rows l % 8 (a) and 8 + l % 8 (b), lanes 0 .. 7 of each 16 with
// x's half, lanes 8 .. 15 with y's.
__device__ __forceinline__ void halves(const uint32_t (&x)[4], const uint32_t (&y)[4], uint32_t (&a)[4], uint32_t (&b)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = (uint32_t)__builtin_amdgcn_update_dpp((int)x[i], (int)y[i], 0x128, 0xF, 0xC, false);   // row_ror:8 into lanes 8 .. 15
    b[i] = (uint32_t)__builtin_amdgcn_update_dpp((int)y[i], (int)x[i], 0x128, 0xF, 0x3, false);   // into lanes 0 .. 7
  }
}
__device__ __forceinline__ void swap_rows(const uint32_t (&p)[4], const uint32_t (&q)[4], uint32_t (&x)[4], uint32_t (&y)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto s = __builtin_amdgcn_permlane16_swap(p[i], q[i], false, false);
    x[i] = s[0];
    y[i] = s[1];
  }
}

// bf16 of a subtile: x rows 0 .. 15, y rows 16 .. 31, columns 16 g + 8 h .. + 7
// (g = l / 16 % 2).
__device__ __forceinline__ void regroup_bf16(const v16f& acc, uint32_t (&x)[4], uint32_t (&y)[4]) {
  uint32_t d[8], a[4], b[4];                          // quad q: d[2 q], d[2 q + 1]
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bf16x2 v = __builtin_convertvector((f32x2){acc[2 * i], acc[2 * i + 1]}, bf16x2);
    __builtin_memcpy(&d[i], &v, 4);
  }
  // lane half h: columns 8 h .. + 7 (from quads 0, 1) and 16 + 8 h .. + 7 (from quads 2, 3)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto s = __builtin_amdgcn_permlane32_swap(d[i], d[2 + i], false, false);
    a[i] = s[0];
    a[2 + i] = s[1];
    const auto t = __builtin_amdgcn_permlane32_swap(d[4 + i], d[6 + i], false, false);
    b[i] = t[0];
    b[2 + i] = t[1];
  }
  swap_rows(a, b, x, y);
}

// Two neighbouring 32 x 32 subtiles of bf16, or one (PAIR false: 64-byte pieces).
template <bool PAIR>
__device__ __forceinline__ void store_bf16(uint16_t* out, int64_t ldo, const v16f& acc0, const v16f& acc1, int lane) {
  const int g = (lane >> 4) & 1, h = lane >> 5;
  uint32_t x0[4], y0[4];
  regroup_bf16(acc0, x0, y0);
  if constexpr (PAIR) {
    uint32_t x1[4], y1[4], a[4], b[4];
    regroup_bf16(acc1, x1, y1);
    uint16_t* p = out + (lane & 7) * ldo + 32 * ((lane >> 3) & 1) + 16 * g + 8 * h;
    halves(x0, x1, a, b);
    put16<true>(p, a);
    put16<true>(p + 8 * ldo, b);
    halves(y0, y1, a, b);
    put16<true>(p + 16 * ldo, a);
    put16<true>(p + 24 * ldo, b);
  } else {
    uint16_t* p = out + (lane & 15) * ldo + 16 * g + 8 * h;
    put16<false>(p, x0);
    put16<false>(p + 16 * ldo, y0);
  }
}

// A 32 x 32 subtile of fp32: quads 2 u and 2 u + 1 trade 16-lane rows (u = 0, 1:
// the halves of a line).
__device__ __forceinline__ void store_f32(float* out, int64_t ldo, const v16f& acc, int lane) {
  const int g = (lane >> 4) & 1, h = lane >> 5;
  uint32_t x[2][4], y[2][4], a[4], b[4];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint32_t p[4], q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = __float_as_uint(acc[8 * u + i]);
      q[i] = __float_as_uint(acc[8 * u + 4 + i]);
    }
    swap_rows(p, q, x[u], y[u]);
  }
  float* p = out + (lane & 7) * ldo + 16 * ((lane >> 3) & 1) + 8 * g + 4 * h;
  halves(x[0], x[1], a, b);
  put16<true>(p, a);
  put16<true>(p + 8 * ldo, b);
  halves(y[0], y[1], a, b);
  put16<true>(p + 16 * ldo, a);
  put16<true>(p + 24 * ldo, b);
}

// A subtile that is cut off by the output's edge, or unaligned rows: element by
// element.
template <bool F32>
__device__ __forceinline__ void store_edge(const MxGemmArgs& p, int64_t base, int64_t m0, int64_t m_end, int64_t n0,
                                           const v16f& acc, int lane) {
  const int64_t row = m0 + (lane & 31);
  if (row >= m_end) return;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int64_t col = n0 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
    if (col < p.n) {
      if constexpr (F32) static_cast<float*>(p.out)[base + row * p.ldo + col] = acc[r];
      else static_cast<uint16_t*>(p.out)[base + row * p.ldo + col] = bf16_bits(acc[r]);
    }
  }
}

template <int MODE, bool F32, int TM, int TN, int NST, bool SPLIT>
__global__ __launch_bounds__(SPLIT ? 512 : 256) void mx_tile_kernel(MxGemmArgs p, int vec_ok) {
  using C = TileCfg<TM, TN>;
  __shared__ __attribute__((aligned(16))) uint8_t smem[NST * C::kStage];
  __shared__ MxTables tab;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave_m = wave & 1, wave_n = wave >> 1;
  const int r32 = lane & 31, h = lane >> 5;

  if constexpr (MODE != MX_DENSE) {
    int64_t lo = 0, hi = 0;
    if (tid < p.groups) group_range(p.row_off, tid, MODE == MX_ROWS ? p.m : (int64_t)p.chunks * 256, lo, hi);
    if (tid < 256) {
      tab.lo[tid] = (int)(MODE == MX_ROWS ? lo : lo / 256);
      tab.hi[tid] = (int)(MODE == MX_ROWS ? hi : hi / 256);
    }
    if constexpr (MODE == MX_ROWS) {
      const int mine = (int)((hi - lo + C::kBM - 1) / C::kBM);
      int sum = mine;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(sum, d);
        if (lane >= d) sum += v;
      }
      __shared__ int wsum[8];
      if (lane == 63) wsum[wave] = sum;
      __syncthreads();
      for (int w = 0; w < wave; ++w) sum += wsum[w];
      if (tid < 256) tab.before[tid + 1] = sum;
      if (tid == 0) tab.before[0] = 0;
    }
    __syncthreads();
  }
  const MxWalk<MODE, TM, TN> wk(p, tab);
  if (wk.mine == 0) return;                                   // uniform
  // Loads a wave has in flight beyond the next step's when a step's barrier is
  // reached; half the waves bring no scales of a small tile.
  auto left = [](bool scales, auto stages) {
    constexpr int n = decltype(stages)::value;
    if (scales) wait_loads_left<n * C::kParts>();
    else wait_loads_left<n * (C::kParts - 1)>();
  };
  MxLoader<MODE, TM, TN> ld(p, wk, lds_addr(smem), wave & 3, lane);
  const bool scales = ld.brings_scales();
  auto wait_next = [&] { left(scales, std::integral_constant<int, NST - 2>{}); };
  if (!SPLIT || wave >= 4) {
#pragma unroll
    for (int st = 0; st < NST; ++st) {
#pragma unroll
      for (int q = 0; q < C::kParts; ++q) ld.part(q, st);
      ld.advance();
    }
    left(scales, std::integral_constant<int, NST - 1>{});
  }
  __syncthreads();
  if (SPLIT && wave >= 4) {
    // a loading wave: the compute waves' barriers, each followed by the loads into the stage that it has freed
    int cs = 0;
#pragma clang loop unroll(disable)
    for (int tk = 0; tk < wk.mine; ++tk) {
      const int nc = wk.tile(tk).nc;
#pragma clang loop unroll(disable)
      for (int c = 0; c < nc; ++c) {
        wait_next();
        __syncthreads();
#pragma unroll
        for (int q = 0; q < C::kParts; ++q) ld.part(q, cs);
        ld.advance();
        cs = cs + 1 < NST ? cs + 1 : 0;
      }
    }
    wait_loads_left<0>();                                     // the repeated loads land before the LDS is released
    return;
  }

  // LDS offset of this lane's codes of slice t in a 32-row subtile: logical slot 4 h + t
  uint32_t off[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) off[t] = r32 * 128 + (((4 * h + t) ^ swz(r32)) * 16);
  auto frag = [&](const uint8_t* base, int t) { return *reinterpret_cast<const v4i*>(base + off[t]); };
  auto a_frag = [&](const uint8_t* st, int i, int t) { return frag(st + (wave_m * TM + i) * 32 * 128, t); };
  auto b_frag = [&](const uint8_t* st, int j, int t) { return frag(st + C::kBOff + (wave_n * TN + j) * 32 * 128, t); };
  auto a_scale = [&](const uint8_t* st, int i) {
    return *reinterpret_cast<const int*>(st + C::kSaOff + ((wave_m * TM + i) * 32 + r32) * 8 + 4 * h);
  };
  auto b_scale = [&](const uint8_t* st, int j) {
    return *reinterpret_cast<const int*>(st + C::kSbOff + ((wave_n * TN + j) * 32 + r32) * 8 + 4 * h);
  };

  v4i af[4][TM], bf[4][TN];
  int ea[TM], eb[TN], ean[TM], ebn[TN];
#pragma unroll
  for (int t = 0; t < 3; ++t) {
#pragma unroll
    for (int i = 0; i < TM; ++i) af[t][i] = a_frag(smem, i, t);
#pragma unroll
    for (int j = 0; j < TN; ++j) bf[t][j] = b_frag(smem, j, t);
  }
#pragma unroll
  for (int i = 0; i < TM; ++i) ea[i] = a_scale(smem, i);
#pragma unroll
  for (int j = 0; j < TN; ++j) eb[j] = b_scale(smem, j);
  __builtin_amdgcn_s_waitcnt(0xC07F);                         // lgkmcnt(0)

  v16f acc[TM][TN];
  constexpr int kNT = TM * TN, kReads = TM + TN;
  int cs = 0;                                                  // the step's stage
  auto step = [&](bool wait_loads) {
    const int ns = cs + 1 < NST ? cs + 1 : 0;
    const uint8_t* st = smem + cs * C::kStage;
    const uint8_t* nst = smem + ns * C::kStage;
    for_each_const([&](auto tc) {
      constexpr int t = decltype(tc)::value / kNT, u = decltype(tc)::value % kNT;
      constexpr int i = u / TN, j = u % TN;
      mfma_slice<t, (TM * TN < 8)>(acc[i][j], bf[t][j], af[t][i], eb[j], ea[i]);
      // the fragments due in this slice, spread over its first MFMAs: slice 3 of this step (t = 0), else slice t - 1 of
      // the next
      constexpr int rs = (t + 3) & 3;
      constexpr int kSpread = kNT / 2 < 1 ? 1 : kNT / 2;      // reads within the first half of the slice
#pragma unroll
      for (int q = 0; q < kReads; ++q) {
        if (q * kSpread / kReads == u) {
          const uint8_t* from = t == 0 ? st : nst;
          if (q < TM) af[rs][q] = a_frag(from, q, rs);
          else bf[rs][q - TM] = b_frag(from, q - TM, rs);
        }
      }
      if constexpr (t == 0 && u == kNT - 1) {
        __builtin_amdgcn_s_waitcnt(0xC07F);                   // slice 3 has been read
        if (!SPLIT && (NST > 2 || wait_loads)) wait_next();
        __syncthreads();
#pragma unroll
        for (int q = 0; q < TM; ++q) ean[q] = a_scale(nst, q);
#pragma unroll
        for (int q = 0; q < TN; ++q) ebn[q] = b_scale(nst, q);
      }
      // the cursor's loads over slices 1 .. 3
      if constexpr (t >= 1 && !SPLIT) {
        constexpr int at = (t - 1) * kNT + u, slots = 3 * kNT;
#pragma unroll
        for (int q = 0; q < C::kParts; ++q)
          if (q * slots / C::kParts == at) ld.part(q, cs);
      }
      if constexpr (t == 3 && u == kNT - 1 && !SPLIT) ld.advance();
      __builtin_amdgcn_sched_barrier(0);
    }, std::make_integer_sequence<int, 4 * kNT>{});
#pragma unroll
    for (int q = 0; q < TM; ++q) ea[q] = ean[q];
#pragma unroll
    for (int q = 0; q < TN; ++q) eb[q] = ebn[q];
    exponents_ready();
    cs = ns;
  };

#pragma clang loop unroll(disable)
  for (int tk = 0; tk < wk.mine; ++tk) {
    const MxTile cur = wk.tile(tk);
    const int nc = cur.nc;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    exponents_ready();
#pragma clang loop unroll(disable)
    for (int c = 0; c < nc; ++c) step(c != 0 || tk == 0);
    mfma_results_ready();
    if constexpr (!SPLIT) wait_loads_left<0>();               // the loads the next tile's first step reads
    const MxTile done = wk.tile(tk);
    const int el = lane_fresh();
    const int64_t base = MODE == MX_K ? (int64_t)done.e * p.m * p.ldo : 0;
    // the subtiles' registers are read where they are stored, not all at once (the asm statements)
    constexpr int kPair = !F32 && TN % 2 == 0 ? 2 : 1;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; j += kPair) {
        const int64_t m0 = done.m0 + (wave_m * TM + i) * 32, n0 = done.n0 + (wave_n * TN + j) * 32;
        asm volatile("" : "+a"(acc[i][j]));
        if constexpr (kPair == 2) asm volatile("" : "+a"(acc[i][j + 1]));
        if (vec_ok && m0 + 32 <= done.m_end && n0 + 32 * kPair <= p.n) {
          if constexpr (F32) store_f32(static_cast<float*>(p.out) + base + m0 * p.ldo + n0, p.ldo, acc[i][j], el);
          else store_bf16<kPair == 2>(static_cast<uint16_t*>(p.out) + base + m0 * p.ldo + n0, p.ldo, acc[i][j],
                                      acc[i][j + kPair - 1], el);
        } else {
#pragma unroll
          for (int k = 0; k < kPair; ++k) store_edge<F32>(p, base, m0, done.m_end, n0 + 32 * k, acc[i][j + k], el);
        }
      }
  }
  if constexpr (!SPLIT) wait_loads_left<0>();                 // the repeated loads land before the LDS is released
}

template <int MODE, bool F32, int TM, int TN, int NST, bool SPLIT>
hipError_t run_tile(const MxGemmArgs& p, hipStream_t st) {
  using C = TileCfg<TM, TN>;
  constexpr int kEsz = F32 ? 4 : 2;
  const int64_t tm = (p.m + C::kBM - 1) / C::kBM + (MODE == MX_ROWS ? p.groups : 0);
  const int64_t tiles = tm * ((p.n + C::kBN - 1) / C::kBN) * (MODE == MX_K ? p.groups : 1);
  const int64_t cus = 256 * (160 * 1024 / (C::kStage * NST + (MODE == MX_DENSE ? 0 : 4096)));
  const unsigned grid = (unsigned)(tiles < cus ? tiles : cus);
  const int vec = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && p.ldo * kEsz % 16 == 0 && p.m * p.ldo * kEsz % 16 == 0;
  mx_tile_kernel<MODE, F32, TM, TN, NST, SPLIT><<<grid, SPLIT ? 512 : 256, 0, st>>>(p, vec);
  return hipGetLastError();
}

template <int MODE, bool F32>
hipError_t run(const MxGemmArgs& p, hipStream_t st) {
  const MxPick pick = mx_pick((MxMode)MODE, p.groups, p.m, p.n, p.chunks);
  switch (pick.tiling) {
    case 1: return run_tile<MODE, F32, 1, 1, 3, true>(p, st);
    case 2: return run_tile<MODE, F32, 1, 2, 3, true>(p, st);
    case 3: return pick.deep ? run_tile<MODE, F32, 2, 2, 3, true>(p, st) : run_tile<MODE, F32, 2, 2, 2, false>(p, st);
    case 4: return run_tile<MODE, F32, 2, 4, 2, false>(p, st);
    case 5: return run_tile<MODE, F32, 4, 4, 2, false>(p, st);
  }
  const unsigned mt = (unsigned)((p.m + 31) / 32) + (MODE == MX_ROWS ? (unsigned)p.groups : 0u);
  const dim3 grid((unsigned)((p.n + 31) / 32) * mt, MODE == MX_K ? (unsigned)p.groups : 1u);
  mx_stream_kernel<MODE, F32, 4><<<grid, 64 * 4, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_mxfp4(const MxGemmArgs& p, MxMode mode, bool f32_out, hipStream_t st) {
  switch (mode) {
    case MX_DENSE: return f32_out ? run<MX_DENSE, true>(p, st) : run<MX_DENSE, false>(p, st);
    case MX_ROWS: return f32_out ? run<MX_ROWS, true>(p, st) : run<MX_ROWS, false>(p, st);
    default: return f32_out ? run<MX_K, true>(p, st) : run<MX_K, false>(p, st);
  }
}

}  // namespace fp8bq
