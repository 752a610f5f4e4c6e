// Routing of tokens to experts: the dispatch plan (counts, offsets, stable row
// order) and the router's balance loss with its gradient. Definitions:
// include/fp8bq.h. No floating-point atomics: every sum has a fixed order.
#include "../../include/fp8bq.h"
#include "lanes.h"
#include "mxfp4.h"

namespace fp8bq {
namespace {

// ---------------------------------------------------------------------------
// Dispatch plan: a stable counting sort of the choices by expert. Each block
// owns a contiguous piece of the flattened choices. Up to one piece it is one
// launch; with more, a first launch writes each piece's histogram to the
// workspace and every block of the second adds up what comes before it (at
// most 256 x 256 counts from the cache; four threads per expert share them).
// Within a block, wave w owns a contiguous sixteenth, walks it 64 choices at a
// time (four loads in flight) and ranks equal experts by eight ballots over
// the expert's bits, so that the order is that of the tokens whatever runs
// when. Bound by latency: 2048 choices are a handful of dependent loads and
// barriers, 4.8 us; 131072 take 10.2 in two launches (their 0.5 MB would be read
// in 0.1), 5.6 and 9.6 behind a prompt's other kernels.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanPiece = 4096;

struct PlanArgs {
  const int32_t* idx;
  int tokens, topk;
  int64_t ldidx;
  int groups, pad, cap;
  int piece;                         // choices per block, a multiple of 4096
  int32_t *counts, *row_off, *src, *pos, *ws;
};

// Experts of choices i0 + 64 u + lane (u = 0 .. 3), -1 for dropped ones and past end.
__device__ __forceinline__ void choices4(const PlanArgs& p, int i0, int end, int (&e)[4]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = i0 + 64 * u + lane;
    e[u] = -1;
    if (i < end) {
      const int t = i / p.topk;
      e[u] = p.ldidx == p.topk ? p.idx[i] : p.idx[(int64_t)t * p.ldidx + (i - t * p.topk)];
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) e[u] = e[u] >= 0 && e[u] < p.groups ? e[u] : -1;
}

__global__ __launch_bounds__(kPlanThreads) void moe_histogram_kernel(PlanArgs p) {
  __shared__ int hist[256];
  const int t = threadIdx.x;
  if (t < 256) hist[t] = 0;
  __syncthreads();
  const int total = p.tokens * p.topk;
  const int lo = blockIdx.x * p.piece, hi = min(lo + p.piece, total);
  for (int i0 = lo + (t >> 6) * 256; i0 < hi; i0 += kPlanWaves * 256) {
    int e[4];
    choices4(p, i0, hi, e);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (e[u] >= 0) atomicAdd(&hist[e[u]], 1);
  }
  __syncthreads();
  if (t < 256) p.ws[blockIdx.x * 256 + t] = hist[t];
}

__global__ __launch_bounds__(kPlanThreads) void moe_place_kernel(PlanArgs p) {
  __shared__ int next[kPlanWaves][256];   // choices of (wave, expert), then the next free row
  __shared__ int sums[2][4][256];         // choices before this block and in all, by quarter of the blocks
  __shared__ int ends[256];               // end of each expert's padded rows
  __shared__ int filled[256];             // end of its real rows
  __shared__ int wtotal[4];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int total = p.tokens * p.topk;
  const int nb = gridDim.x, blk = blockIdx.x;
#pragma unroll
  for (int w = 0; w < kPlanWaves / 4; ++w) next[w * 4 + (t >> 8)][t & 255] = 0;

  // what the other blocks have
  int before = 0, all = 0;
  if (nb > 1) {
#pragma unroll 8
    for (int b = t >> 8; b < nb; b += 4) {
      const int c = p.ws[b * 256 + (t & 255)];
      before += b < blk ? c : 0;
      all += c;
    }
    sums[0][t >> 8][t & 255] = before;
    sums[1][t >> 8][t & 255] = all;
  }
  __syncthreads();

  // this block's choices per wave and expert
  const int lo = blk * p.piece, hi = min(lo + p.piece, total);
  const int part = p.piece / kPlanWaves;
  const int wlo = lo + wave * part, whi = min(wlo + part, hi);
  int first_e[4] = {-1, -1, -1, -1};                 // the first 256 stay in registers
  for (int i0 = wlo; i0 < whi; i0 += 256) {
    int e[4];
    choices4(p, i0, whi, e);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (i0 == wlo) first_e[u] = e[u];
      if (e[u] >= 0) atomicAdd(&next[wave][e[u]], 1);
    }
  }
  __syncthreads();

  // thread e < 256: offsets of expert e, by a scan over the waves' 64 experts each
  int padded = 0, scan = 0;
  if (t < 256) {
    if (nb > 1) {
      before = sums[0][0][t] + sums[0][1][t] + sums[0][2][t] + sums[0][3][t];
      all = sums[1][0][t] + sums[1][1][t] + sums[1][2][t] + sums[1][3][t];
    } else {
#pragma unroll
      for (int w = 0; w < kPlanWaves; ++w) all += next[w][t];
    }
    padded = (all + p.pad - 1) / p.pad * p.pad;
    scan = padded;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(scan, d);
      if (lane >= d) scan += v;
    }
    if (lane == 63) wtotal[wave] = scan;
  }
  __syncthreads();
  if (t < 256) {
    for (int w = 0; w < wave; ++w) scan += wtotal[w];
    const int first = scan - padded;
    ends[t] = scan;
    filled[t] = first + all;
    int at = first + before;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = next[w][t];
      next[w][t] = at;
      at += c;
    }
    if (blk == 0) {
      if (t < p.groups) {
        p.counts[t] = all;
        p.row_off[t] = first;
      }
      if (t == 255) p.row_off[p.groups] = scan;
    }
  }
  __syncthreads();

  // rows without a token: the padding of the experts dealt to this wave, and
  // this block's share of what lies behind the last expert
  for (int e = blk + nb * wave; e < p.groups; e += nb * kPlanWaves)
    for (int r = filled[e] + lane; r < ends[e]; r += 64) p.src[r] = -1;
  for (int64_t r = (int64_t)ends[255] + blk * kPlanThreads + t; r < p.cap; r += (int64_t)nb * kPlanThreads)
    p.src[r] = FP8BQ_ROW_UNUSED;

  // places, in order
  for (int i0 = wlo; i0 < whi; i0 += 256) {
    int e4[4] = {first_e[0], first_e[1], first_e[2], first_e[3]};
    if (i0 != wlo) choices4(p, i0, whi, e4);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + 64 * u + lane, e = e4[u];
      uint64_t same = __ballot(e >= 0);
#pragma unroll
      for (int bit = 0; bit < 8; ++bit) {
        const uint64_t m = __ballot((e >> bit) & 1);
        same &= ((e >> bit) & 1) ? m : ~m;
      }
      const uint64_t below = same & ((1ull << lane) - 1);
      int row = -1;
      if (e >= 0) row = next[wave][e] + __popcll(below);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // every lane has read before the first of its kind adds
      if (e >= 0 && below == 0) next[wave][e] += __popcll(same);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (i < whi) {
        p.pos[i] = row;
        if (row >= 0) p.src[row] = i / p.topk;
      }
    }
  }
}

}  // namespace

hipError_t launch_moe_plan(const int32_t* idx, int tokens, int topk, int64_t ldidx, int groups, int pad,
                           int32_t* counts, int32_t* row_off, int32_t* src, int cap, int32_t* pos, int32_t* ws,
                           hipStream_t stream) {
  PlanArgs p{idx, tokens, topk, ldidx, groups, pad, cap, kPlanPiece, counts, row_off, src, pos, ws};
  const int total = tokens * topk;
  if ((total + kPlanPiece - 1) / kPlanPiece > kMoePlanMaxBlocks)
    p.piece = ((total + kMoePlanMaxBlocks - 1) / kMoePlanMaxBlocks + kPlanPiece - 1) / kPlanPiece * kPlanPiece;
  const int nb = (total + p.piece - 1) / p.piece;
  if (nb > 1) {
    moe_histogram_kernel<<<nb, kPlanThreads, 0, stream>>>(p);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  moe_place_kernel<<<nb, kPlanThreads, 0, stream>>>(p);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Balance loss. A wave takes a token (its experts over the lanes, so that a
// softmax is two reductions in registers), two tokens' loads in flight. 16384
// tokens of 256 experts (fp32, 4 sequences): 7.9 us the sums, 5.8 the joining of
// the pieces, 10.7 the gradient, where the bytes would take 3.3, 0.1 and 6.5: an
// empty kernel takes 2.5, and a wave has but four tokens, one after the other.
// Two tokens' arithmetic side by side without branches was slower by 10%.
// ---------------------------------------------------------------------------
namespace {

template <int T> struct Logit { using type = uint16_t; };
template <> struct Logit<FP8BQ_FP32> { using type = float; };
template <int T>
__device__ __forceinline__ float logit_value(typename Logit<T>::type b) {
  if constexpr (T == FP8BQ_FP32) {
    return b;
  } else if constexpr (T == FP8BQ_BF16) {
    return __uint_as_float((uint32_t)b << 16);
  } else {
    _Float16 h;
    __builtin_memcpy(&h, &b, 2);
    return (float)h;
  }
}
template <int T>
__device__ __forceinline__ typename Logit<T>::type logit_round(float v) {
  typename Logit<T>::type r;
  if constexpr (T == FP8BQ_FP32) {
    r = v;
  } else if constexpr (T == FP8BQ_BF16) {
    const __bf16 b = (__bf16)v;
    __builtin_memcpy(&r, &b, 2);
  } else {
    const _Float16 h = (_Float16)v;
    __builtin_memcpy(&r, &h, 2);
  }
  return r;
}

// Which experts a lane holds: VPL neighbours (PACK: the experts are a multiple
// of VPL and rows are aligned, a lane moves them in one or a few wide accesses),
// or every 64th.
template <int VPL, bool PACK>
__device__ __forceinline__ int expert_of(int lane, int i) { return PACK ? lane * VPL + i : lane + 64 * i; }

template <int T, int VPL, bool PACK>
__device__ __forceinline__ void load_logits(const void* base, int64_t row, int experts, float (&v)[VPL]) {
  using E = typename Logit<T>::type;
  const int lane = threadIdx.x & 63;
  const E* p = static_cast<const E*>(base) + row;
  E raw[VPL];
  if constexpr (PACK) {
    constexpr int kBytes = VPL * sizeof(E);
    if (lane * VPL < experts) __builtin_memcpy(raw, __builtin_assume_aligned(p + lane * VPL, kBytes < 16 ? kBytes : 16), kBytes);
    else __builtin_memset(raw, 0, kBytes);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) raw[i] = lane + 64 * i < experts ? p[lane + 64 * i] : (E)0;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) v[i] = logit_value<T>(raw[i]);
}
template <int T, int VPL, bool PACK>
__device__ __forceinline__ void store_logits(void* base, int64_t row, int experts, const float (&v)[VPL]) {
  using E = typename Logit<T>::type;
  const int lane = threadIdx.x & 63;
  E* p = static_cast<E*>(base) + row;
  E raw[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) raw[i] = logit_round<T>(v[i]);
  if constexpr (PACK) {
    constexpr int kBytes = VPL * sizeof(E);
    if (lane * VPL < experts) __builtin_memcpy(__builtin_assume_aligned(p + lane * VPL, kBytes < 16 ? kBytes : 16), raw, kBytes);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 64 * i < experts) p[lane + 64 * i] = raw[i];
  }
}

// e^x for x <= 0: 2^t of t = x log2(e), times 1 + what t's rounding left over
// (which is up to |x| 2^-24 of the result), log2(e) and ln 2 being the
// mathematical constants to double precision and the low part of log2(e) what
// its rounding to float leaves.
constexpr double kLog2E = 1.44269504088896340736, kLn2 = 0.69314718055994530942;
constexpr float kLog2EHigh = (float)kLog2E, kLog2ELow = (float)(kLog2E - (double)kLog2EHigh);
__device__ __forceinline__ float exp_neg(float x) {
  const float t = x * kLog2EHigh;
  const float rest = __builtin_fmaf(x, kLog2EHigh, -t) + x * kLog2ELow;
  const float r = __builtin_amdgcn_exp2f(t);
  return t < -126.f ? 0.f : __builtin_fmaf(r, rest * (float)kLn2, r);
}

// Tokens of sequence s, clamped into the batch; s == sequences: nothing here.
__device__ __forceinline__ void seq_range(const MoeBalanceArgs& a, int s, int64_t& lo, int64_t& hi) {
  lo = 0;
  hi = a.tokens;
  if (a.seq_off) {
    lo = min(max((int64_t)a.seq_off[s], (int64_t)0), a.tokens);
    hi = min(max((int64_t)a.seq_off[s + 1], lo), a.tokens);
  }
}

// One token's row: a lane's logits and its choices l, l + 64, ... (the first of
// them here, the rest where topk > 64). Loaded for two tokens at a time,
// before anything is used.
template <int T, int VPL, bool PACK>
struct TokenRow {
  float v[VPL];
  int first;
  __device__ __forceinline__ void load(const MoeBalanceArgs& a, int64_t t) {
    const int lane = threadIdx.x & 63;
    first = lane < a.topk ? a.idx[t * a.ldidx + lane] : -1;
    load_logits<T, VPL, PACK>(a.logits, t * a.ldl, a.experts, v);
  }
};

// Whether a token has a choice inside [0, experts) (all lanes of the wave);
// each such choice is given to count(e).
template <class F>
__device__ __forceinline__ bool real_token(const MoeBalanceArgs& a, int64_t t, int first, F&& count) {
  bool any = first >= 0 && first < a.experts;
  if (any) count(first);
  for (int j = 64 + (threadIdx.x & 63); j < a.topk; j += 64) {
    const int e = a.idx[t * a.ldidx + j];
    if (e >= 0 && e < a.experts) {
      any = true;
      count(e);
    }
  }
  return __any(any);
}

// p of a token. v: logits in, p out; open: 1 - sigmoid (SIGMOID).
template <bool SIG, int VPL, bool PACK>
__device__ __forceinline__ void probabilities(float (&v)[VPL], float (&open)[VPL], int experts) {
  const int lane = threadIdx.x & 63;
  float sum = 0.f;
  if constexpr (SIG) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      // sigmoid and its complement from the same exponential, neither by subtraction
      const float z = exp_neg(-fabsf(v[i])), inv = 1.f / (1.f + z);
      const float big = inv, small = z * inv;
      const bool in = expert_of<VPL, PACK>(lane, i) < experts;
      open[i] = v[i] >= 0.f ? small : big;
      v[i] = in ? (v[i] >= 0.f ? big : small) : 0.f;
      sum += v[i];
    }
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, expert_of<VPL, PACK>(lane, i) < experts ? v[i] : -INFINITY);
    m = wave_max(m);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      // -inf is a masked expert, also where all are (m = -inf); a NaN stays one, also where nothing else is there
      v[i] = expert_of<VPL, PACK>(lane, i) < experts && v[i] != -INFINITY ? exp_neg(v[i] - m) : 0.f;
      sum += v[i];
    }
  }
  sum = wave_sum(sum);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;      // NaN goes to every expert
#pragma unroll
  for (int i = 0; i < VPL; ++i) v[i] *= inv;
}

constexpr int kBalWaves = 16;     // of the forward kernel: few, large partial results
constexpr int kGradWaves = 4;

// Pieces a sequence is cut into for blocks of `waves` waves: about 4096 waves
// in all, at least two tokens each.
int balance_pieces(int64_t tokens, int64_t sequences, int waves) {
  int64_t c = 4096 / waves / sequences;
  const int64_t per = (tokens / sequences + 2 * waves - 1) / (2 * waves);
  c = c < per ? c : per;
  return (int)(c < 1 ? 1 : c > 256 ? 256 : c);
}

// Workspace: per (sequence, piece): experts floats (sums of p), experts ints
// (counts), one int (real tokens); then one float per (sequence, 64 experts),
// its part of the loss, and the ticket.
struct BalanceWs {
  float* psum;
  int32_t* cnt;
  int32_t* real;
  float* part;
  int32_t* ticket;
};
__host__ __device__ inline BalanceWs balance_ws(void* ws, int64_t experts, int64_t sequences, int64_t pieces) {
  BalanceWs w;
  const int64_t rows = sequences * pieces;
  w.psum = static_cast<float*>(ws);
  w.cnt = reinterpret_cast<int32_t*>(w.psum + rows * experts);
  w.real = w.cnt + rows * experts;
  w.part = reinterpret_cast<float*>(w.real + rows);
  w.ticket = reinterpret_cast<int32_t*>(w.part + sequences * ((experts + 63) / 64));
  return w;
}

// Block (piece, sequence): a wave per token; a lane sums p of its experts in
// registers, the waves meet in LDS.
template <int T, bool SIG, int VPL, bool PACK>
__global__ __launch_bounds__(64 * kBalWaves) void balance_partial_kernel(MoeBalanceArgs a, int pieces, void* ws) {
  __shared__ float sums[kBalWaves][VPL * 64];
  __shared__ int hist[VPL * 64];
  __shared__ int reals[kBalWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const BalanceWs w = balance_ws(ws, a.experts, a.sequences, pieces);
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *w.ticket = 0;
  for (int i = tid; i < VPL * 64; i += 64 * kBalWaves) hist[i] = 0;
  __syncthreads();
  int64_t lo, hi;
  seq_range(a, blockIdx.y, lo, hi);
  const int64_t per = (hi - lo + pieces - 1) / pieces;
  const int64_t t0 = lo + (int64_t)blockIdx.x * per, t1 = min(t0 + per, hi);
  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.f;
  int real = 0;
  auto take = [&](TokenRow<T, VPL, PACK>& row, int64_t t) {
    if (!real_token(a, t, row.first, [&](int e) { atomicAdd(&hist[e], 1); })) return;
    ++real;
    float open[VPL];
    probabilities<SIG, VPL, PACK>(row.v, open, a.experts);
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] += row.v[i];
  };
  for (int64_t t = t0 + wave; t < t1; t += 2 * kBalWaves) {
    TokenRow<T, VPL, PACK> x, y;
    x.load(a, t);
    const bool two = t + kBalWaves < t1;             // uniform in the wave
    if (two) y.load(a, t + kBalWaves);
    take(x, t);
    if (two) take(y, t + kBalWaves);
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) sums[wave][expert_of<VPL, PACK>(lane, i)] = acc[i];
  if (lane == 0) reals[wave] = real;
  __syncthreads();
  const int64_t row = (int64_t)blockIdx.y * pieces + blockIdx.x;
  for (int e = tid; e < a.experts; e += 64 * kBalWaves) {
    float s = sums[0][e];
#pragma unroll
    for (int v = 1; v < kBalWaves; ++v) s += sums[v][e];
    w.psum[row * a.experts + e] = s;
    w.cnt[row * a.experts + e] = hist[e];
  }
  if (tid == 0) {
    int s = 0;
    for (int v = 0; v < kBalWaves; ++v) s += reals[v];
    w.real[row] = s;
  }
}

// Block (64 experts, sequence) adds up the pieces: wave w takes pieces w,
// w + 16, ... (a lane an expert), the waves meet in LDS in their order. It
// writes counts and real, and its part of the loss; the last block to finish
// adds the parts in order.
constexpr int kFinalWaves = 16;
__global__ __launch_bounds__(64 * kFinalWaves) void balance_final_kernel(MoeBalanceArgs a, int pieces, void* ws,
                                                                         float* loss, int32_t* counts,
                                                                         int32_t* real_out) {
  __shared__ float psum[kFinalWaves][64];
  __shared__ int csum[kFinalWaves][64], rsum[kFinalWaves];
  __shared__ double red[64 * kFinalWaves];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, s = blockIdx.y;
  const int e = blockIdx.x * 64 + lane;
  const BalanceWs w = balance_ws(ws, a.experts, a.sequences, pieces);
  const int64_t row0 = (int64_t)s * pieces;
  float p = 0.f;
  int n = 0, real = 0;
#pragma unroll 4
  for (int c = wave; c < pieces; c += kFinalWaves) {
    if (e < a.experts) {
      p += w.psum[(row0 + c) * a.experts + e];
      n += w.cnt[(row0 + c) * a.experts + e];
    }
    real += w.real[row0 + c];                          // the same on every lane
  }
  psum[wave][lane] = p;
  csum[wave][lane] = n;
  if (lane == 0) rsum[wave] = real;
  __syncthreads();
  if (wave == 0) {
    double ps = 0.0;
    int ns = 0, rs = 0;
#pragma unroll
    for (int v = 0; v < kFinalWaves; ++v) {
      ps += (double)psum[v][lane];
      ns += csum[v][lane];
      rs += rsum[v];
    }
    if (e < a.experts) counts[(int64_t)s * a.experts + e] = ns;
    double dot = ps * ns;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d);
    if (lane == 0) {
      if (blockIdx.x == 0) real_out[s] = rs;
      const double part = rs ? dot * a.experts / ((double)a.topk * rs * rs) : 0.0;
      __hip_atomic_store(&w.part[(int64_t)s * gridDim.x + blockIdx.x], (float)part, __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
      const int blocks = (int)(gridDim.x * gridDim.y);
      last = __hip_atomic_fetch_add(w.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == blocks - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  double sum = 0.0;
  for (int i = tid; i < (int)(gridDim.x * gridDim.y); i += 64 * kFinalWaves)
    sum += (double)__hip_atomic_load(&w.part[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  red[tid] = sum;
  __syncthreads();
  for (int d = 32 * kFinalWaves; d >= 1; d >>= 1) {
    if (tid < d) red[tid] += red[tid + d];
    __syncthreads();
  }
  if (tid == 0) *loss = (float)(red[0] * (double)a.coef / a.sequences);
}

// The batch's table of offsets as a wave sees it; up to 63 sequences' offsets sit
// in its lanes from one load.
struct Sequences {
  const int32_t* off;
  int count, mine;
  int64_t tokens;
  __device__ __forceinline__ explicit Sequences(const MoeBalanceArgs& a)
      : off(a.seq_off), count(a.sequences), mine(0x7FFFFFFF), tokens(a.tokens) {
    const int lane = threadIdx.x & 63;
    if (off && count < 64 && lane <= count) mine = off[lane];
  }
  // Offset s, within the batch.
  __device__ __forceinline__ int64_t at(int s) const {
    if (!off) return s == 0 ? 0 : tokens;
    const int64_t v = count < 64 ? __builtin_amdgcn_readlane(mine, s) : off[s];
    return min(max(v, (int64_t)0), tokens);
  }
  // The sequence of token t (0 <= t < tokens): the last one that begins at or
  // before it; -1 before the first, `count` behind the last. end: the first
  // token above t that is not of it. A longer table is searched 64 offsets at a
  // time, the last ones of 64 equal stretches.
  __device__ __forceinline__ int of(int64_t t, int64_t& end) const {
    end = tokens;
    if (!off) return 0;
    int next = 0;                                      // offsets at or before t
    if (count < 64) {
      next = __popcll(__ballot((int64_t)mine <= t));
    } else {
      const int lane = threadIdx.x & 63;
      for (int n = count + 1; n > 0;) {                // the first one above t is among the n from `next` on, or behind
        const int step = (n + 63) / 64, i = lane * step + step - 1;
        const int c = __popcll(__ballot(i < n && (int64_t)off[next + (i < n ? i : 0)] <= t)) * step;
        next += c;
        n = min(step - 1, n - c);
      }
    }
    next = __builtin_amdgcn_readfirstlane(next);
    if (next <= count) end = min(max(at(next), t + 1), tokens);
    return next - 1;
  }
};

// Gradient. Each wave takes a contiguous run of the sequences' tokens, whatever
// their lengths (65536 tokens of 64 experts in 1000 sequences: 19 us where blocks
// of their own for each sequence took 903; 2^20 tokens: 237 against 14417); of
// each sequence that it meets, the lane's coefficients f = dloss * coef / S * experts *
// c / (topk * n^2) stay in registers. p (f - sum p f) is the same for f less any
// constant, the p of a token adding up to 1 (or all 0): the mean count comes off
// as a whole number first, or nearly even loads would leave little but the
// rounding of f. The tokens outside every sequence, which get
// zeros, are dealt out beside that (half of 2^20 tokens outside: 137 us, 198 where
// they were part of the runs).
template <int T, bool SIG, int VPL, bool PACK>
__global__ __launch_bounds__(64 * kGradWaves) void balance_grad_kernel(MoeBalanceArgs a, const float* dloss,
                                                                      const int32_t* counts, const int32_t* real,
                                                                      void* dlogits, int64_t lddl) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Sequences seq(a);
  const int64_t begin = seq.at(0), stop = max(seq.at(a.sequences), begin);
  const int64_t id = (int64_t)blockIdx.x * kGradWaves + wave, waves = (int64_t)gridDim.x * kGradWaves;
  const int64_t run = (stop - begin + waves - 1) / waves, first = begin + id * run, last = min(first + run, stop);
  for (int64_t t = first, end; t < last; t = end) {
    const int s = seq.of(t, end);
    end = min(end, last);
    if (s < 0 || s >= a.sequences) continue;            // only with offsets that decrease
    const float n = (float)max(real[s], 1);
    const float scale = dloss[0] * (a.coef / a.sequences) * ((float)a.experts / ((float)a.topk * n)) / n;
    const int mean = (int)((int64_t)a.topk * real[s] / a.experts);
    float f[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      f[i] = expert_of<VPL, PACK>(lane, i) < a.experts
                 ? scale * (float)(counts[(int64_t)s * a.experts + expert_of<VPL, PACK>(lane, i)] - mean) : 0.f;
    auto take = [&](TokenRow<T, VPL, PACK>& row, int64_t at) {
      const bool ok = real_token(a, at, row.first, [](int) {});
      float (&v)[VPL] = row.v;
      float open[VPL];
      probabilities<SIG, VPL, PACK>(v, open, a.experts);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) dot += v[i] * f[i];
      dot = wave_sum(dot);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        float d = v[i] * (f[i] - dot);
        if constexpr (SIG) d *= open[i];
        v[i] = ok ? d : 0.f;
      }
      store_logits<T, VPL, PACK>(dlogits, at * lddl, a.experts, v);
    };
    for (; t < end; t += 2) {
      TokenRow<T, VPL, PACK> x, y;
      x.load(a, t);
      const bool two = t + 1 < end;                     // uniform in the wave
      if (two) y.load(a, t + 1);
      take(x, t);
      if (two) take(y, t + 1);
    }
  }
  for (int64_t u = id; u < a.tokens - (stop - begin); u += waves) {
    const float zero[VPL] = {};
    store_logits<T, VPL, PACK>(dlogits, (u < begin ? u : stop + (u - begin)) * lddl, a.experts, zero);
  }
}

template <int T, bool SIG, int VPL, bool PACK>
hipError_t run_balance(const MoeBalanceArgs& a, float* loss, int32_t* counts, int32_t* real, void* ws, hipStream_t st) {
  const int pieces = balance_pieces(a.tokens, a.sequences, kBalWaves);
  balance_partial_kernel<T, SIG, VPL, PACK><<<dim3(pieces, a.sequences), 64 * kBalWaves, 0, st>>>(a, pieces, ws);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  balance_final_kernel<<<dim3((a.experts + 63) / 64, a.sequences), 64 * kFinalWaves, 0, st>>>(a, pieces, ws, loss, counts, real);
  return hipGetLastError();
}
template <int T, bool SIG, int VPL, bool PACK>
hipError_t run_grad(const MoeBalanceArgs& a, const float* dloss, const int32_t* counts, const int32_t* real,
                    void* dlogits, int64_t lddl, hipStream_t st) {
  // about 4096 waves, of at least two tokens each
  const int64_t run = a.tokens > 2 * 4096 ? (a.tokens + 4095) / 4096 : 2;
  const unsigned blocks = (unsigned)((a.tokens + run * kGradWaves - 1) / (run * kGradWaves));
  balance_grad_kernel<T, SIG, VPL, PACK><<<blocks, 64 * kGradWaves, 0, st>>>(a, dloss, counts, real, dlogits, lddl);
  return hipGetLastError();
}

// f<T, SIG, VPL, PACK>() for the call's type, score, experts per lane and alignment.
template <int T, bool SIG, int VPL, class F>
hipError_t by_layout(const MoeBalanceArgs& a, const void* also, int64_t also_ld, F&& f) {
  constexpr int kBytes = VPL * (T == FP8BQ_FP32 ? 4 : 2), kAlign = kBytes < 16 ? kBytes : 16;
  constexpr int64_t kElem = T == FP8BQ_FP32 ? 4 : 2;
  if constexpr (VPL > 1) {
    if (a.experts % VPL == 0 && reinterpret_cast<uintptr_t>(a.logits) % kAlign == 0 && a.ldl * kElem % kAlign == 0 &&
        reinterpret_cast<uintptr_t>(also) % kAlign == 0 && also_ld * kElem % kAlign == 0)
      return f.template operator()<T, SIG, VPL, true>();
  }
  return f.template operator()<T, SIG, VPL, false>();
}
template <int T, bool SIG, class F>
hipError_t by_width(const MoeBalanceArgs& a, const void* also, int64_t also_ld, F&& f) {
  if (a.experts <= 64) return by_layout<T, SIG, 1>(a, also, also_ld, f);
  if (a.experts <= 128) return by_layout<T, SIG, 2>(a, also, also_ld, f);
  if (a.experts <= 256) return by_layout<T, SIG, 4>(a, also, also_ld, f);
  if (a.experts <= 512) return by_layout<T, SIG, 8>(a, also, also_ld, f);
  return by_layout<T, SIG, 16>(a, also, also_ld, f);
}
template <class F>
hipError_t by_kind(const MoeBalanceArgs& a, int ltype, bool sigmoid, const void* also, int64_t also_ld, F&& f) {
  switch (ltype) {
    case FP8BQ_BF16:
      return sigmoid ? by_width<FP8BQ_BF16, true>(a, also, also_ld, f) : by_width<FP8BQ_BF16, false>(a, also, also_ld, f);
    case FP8BQ_FP16:
      return sigmoid ? by_width<FP8BQ_FP16, true>(a, also, also_ld, f) : by_width<FP8BQ_FP16, false>(a, also, also_ld, f);
    default:
      return sigmoid ? by_width<FP8BQ_FP32, true>(a, also, also_ld, f) : by_width<FP8BQ_FP32, false>(a, also, also_ld, f);
  }
}
struct Forward {
  const MoeBalanceArgs& a; float* loss; int32_t* counts; int32_t* real; void* ws; hipStream_t st;
  template <int T, bool SIG, int VPL, bool PACK> hipError_t operator()() {
    return run_balance<T, SIG, VPL, PACK>(a, loss, counts, real, ws, st);
  }
};
struct Backward {
  const MoeBalanceArgs& a; const float* dloss; const int32_t* counts; const int32_t* real; void* dlogits; int64_t lddl;
  hipStream_t st;
  template <int T, bool SIG, int VPL, bool PACK> hipError_t operator()() {
    return run_grad<T, SIG, VPL, PACK>(a, dloss, counts, real, dlogits, lddl, st);
  }
};

}  // namespace

int64_t moe_balance_workspace(int64_t tokens, int64_t experts, int64_t sequences) {
  const int64_t rows = sequences * balance_pieces(tokens, sequences, kBalWaves);
  return 4 * (rows * (2 * experts + 1) + sequences * ((experts + 63) / 64) + 1);
}

hipError_t launch_moe_balance(const MoeBalanceArgs& a, int ltype, bool sigmoid, float* loss, int32_t* counts,
                              int32_t* real, void* ws, hipStream_t stream) {
  return by_kind(a, ltype, sigmoid, nullptr, 0, Forward{a, loss, counts, real, ws, stream});
}

hipError_t launch_moe_balance_grad(const MoeBalanceArgs& a, int ltype, bool sigmoid, const float* dloss,
                                   const int32_t* counts, const int32_t* real, void* dlogits, int64_t lddl,
                                   hipStream_t stream) {
  return by_kind(a, ltype, sigmoid, dlogits, lddl, Backward{a, dloss, counts, real, dlogits, lddl, stream});
}

}  // namespace fp8bq
