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
#include "mxfp4.h"

namespace fp8bq {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
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

  const int64_t n0 = (int64_t)blockIdx.x * 32;
  int64_t m0 = (int64_t)blockIdx.y * 32, m_end = min(m0 + 32, p.m);
  const uint8_t* b = p.b;
  const uint8_t* sb = p.sb;
  int64_t out_base = 0;
  int c0 = 0, c1 = p.chunks;
  if constexpr (MODE == MX_ROWS) {
    const RowTile t = find_tile<32>(p.row_off, p.groups, p.m, blockIdx.y);
    if (t.e < 0) return;
    m0 = t.m0;
    m_end = t.m_end;
    b += (int64_t)t.e * p.n * p.ldb;
    sb += (int64_t)t.e * p.chunks * p.ldsb * 8;
  }
  if constexpr (MODE == MX_K) {
    const int e = blockIdx.z;
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
  for (int c = c0 + wave; c < c1; c += WAVES) {
    uint4 av[4], bv[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      bv[t] = *reinterpret_cast<const uint4*>(pb + (int64_t)c * 128 + t * 16);
      av[t] = *reinterpret_cast<const uint4*>(pa + (int64_t)c * 128 + t * 16);
    }
    const int ea = *reinterpret_cast<const int*>(psa + (int64_t)c * p.ldsa * 8);
    const int eb = *reinterpret_cast<const int*>(psb + (int64_t)c * p.ldsb * 8);
    acc = mfma<0>(bv[0], av[0], acc, eb, ea);
    acc = mfma<1>(bv[1], av[1], acc, eb, ea);
    acc = mfma<2>(bv[2], av[2], acc, eb, ea);
    acc = mfma<3>(bv[3], av[3], acc, eb, ea);
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

template <int MODE, bool F32>
hipError_t run(const MxGemmArgs& p, hipStream_t st) {
  constexpr int kWaves = 4;
  const unsigned mt = (unsigned)((p.m + 31) / 32) + (MODE == MX_ROWS ? (unsigned)p.groups : 0u);
  const dim3 grid((unsigned)((p.n + 31) / 32), mt, MODE == MX_K ? (unsigned)p.groups : 1u);
  mx_stream_kernel<MODE, F32, kWaves><<<grid, 64 * kWaves, 0, st>>>(p);
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
