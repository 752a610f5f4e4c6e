// Host-only driver for the entry points of the MXFP4 and routing operators
// (csrc/api_mxfp4.cpp with csrc/api.cpp), built with AddressSanitizer and
// UndefinedBehaviorSanitizer (g++, no GPU code): refusals with sizes up to
// INT64_MAX, and accepted calls through to stand-ins for the launchers that
// check what reaches them. Built and run by tests/test_abi_mxfp4_sanitized.py.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "fp8bq.h"
#include "internal.h"
#include "mxfp4.h"

static int g_launches = 0;

extern "C" hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
extern "C" hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
  std::memset(p, 0, sizeof(*p));
  std::strcpy(p->gcnArchName, "gfx950:sramecc+:xnack-");
  return hipSuccess;
}
extern "C" hipError_t hipGetLastError(void) { return hipSuccess; }
extern "C" const char* hipGetErrorString(hipError_t) { return "stub"; }

namespace fp8bq {
// the FP8 launchers that api.cpp refers to: never reached here
#define UNREACHED { std::abort(); }
hipError_t launch_quant_act_rows(const uint16_t*, int64_t, int64_t, int64_t, uint8_t*, int64_t, float*, int64_t, bool, hipStream_t) UNREACHED
hipError_t launch_quant_act_cols(const uint16_t*, int64_t, int64_t, int64_t, uint8_t*, int64_t, float*, int64_t, bool, hipStream_t) UNREACHED
hipError_t launch_quant_w(const uint16_t*, int64_t, int64_t, int64_t, uint8_t*, int64_t, float*, int64_t, uint8_t*, int64_t, bool, hipStream_t) UNREACHED
hipError_t launch_requant_t(const uint8_t*, int64_t, int64_t, int64_t, const float*, int64_t, uint8_t*, int64_t, float*, int64_t, bool, hipStream_t) UNREACHED
hipError_t launch_cache_e5m6(const uint16_t*, int64_t, int64_t, int64_t, uint8_t*, int64_t, float*, int64_t, hipStream_t) UNREACHED
hipError_t launch_uncache_e5m6(const uint8_t*, int64_t, int64_t, int64_t, const float*, int64_t, uint16_t*, int64_t, hipStream_t) UNREACHED
hipError_t launch_requant_e5m6_t(const uint8_t*, int64_t, int64_t, int64_t, const float*, int64_t, uint8_t*, int64_t, float*, int64_t, hipStream_t) UNREACHED
hipError_t launch_gemm(int, int64_t, int64_t, int64_t, const uint8_t*, int64_t, const float*, int64_t, const uint8_t*, int64_t, const float*, int64_t, void*, int64_t, bool, hipStream_t) UNREACHED
hipError_t launch_gemm_quant(int, int64_t, int64_t, int64_t, const uint8_t*, int64_t, const float*, int64_t, const uint8_t*, int64_t, const float*, int64_t, uint16_t*, int64_t, uint8_t*, int64_t, float*, int64_t, bool, bool, hipStream_t) UNREACHED
hipError_t launch_grouped_gemm(int, const int64_t*, int64_t, int64_t, const uint8_t*, int64_t, const float*, int64_t, const uint8_t*, int64_t, const float*, int64_t, uint16_t*, int64_t, bool, hipStream_t) UNREACHED
hipError_t launch_grouped_gemm_decode(int, const int64_t*, int64_t, int64_t, const uint8_t*, int64_t, const float*, int64_t, const uint8_t*, int64_t, const float*, int64_t, uint16_t*, int64_t, void*, hipStream_t) UNREACHED
int64_t grouped_gemm_decode_workspace(int, const int64_t*, int64_t, int64_t) UNREACHED
hipError_t launch_grouped_gemm_decode_noalloc(int, const int64_t*, int64_t, int64_t, const uint8_t*, int64_t, const float*, int64_t, const uint8_t*, int64_t, const float*, int64_t, uint16_t*, int64_t, hipStream_t) UNREACHED

#define REQUIRE(c) do { if (!(c)) { std::fprintf(stderr, "launcher got: not (%s)\n", #c); std::abort(); } } while (0)
hipError_t launch_quant_mxfp4(const MxQuantArgs& a, int xtype, bool, int32_t* ws, hipStream_t) {
  REQUIRE(a.rows > 0 && a.cols > 0 && a.ldx >= a.cols && xtype >= 0 && xtype <= 2 && (a.q || a.qt));
  REQUIRE((a.rows + 15) / 16 * ((a.cols + 255) / 256) <= (1 << 24) && (a.cols + 255) / 256 <= 16383);
  REQUIRE(!a.q || (a.ldq >= (a.cols + 255) / 256 * 128 && a.lds >= a.rows && a.s));
  REQUIRE(!a.qt || (a.ldqt >= (a.rows + 255) / 256 * 128 && a.ldst >= a.cols && a.st));
  REQUIRE(!ws || (a.src && !a.qt && a.rows >= 2 * a.xrows));
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_dequant_mxfp4(const uint8_t*, int64_t rows, int64_t cols, int64_t ldq, const uint8_t*, int64_t lds, void*,
                                int, int64_t ldy, hipStream_t) {
  REQUIRE(rows > 0 && cols > 0 && ldq >= (cols + 255) / 256 * 128 && lds >= rows && ldy >= cols);
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_gemm_mxfp4(const MxGemmArgs& p, MxMode mode, bool, hipStream_t) {
  REQUIRE(p.m > 0 && p.n > 0 && p.chunks > 0 && p.ldo >= p.n && p.lda < (1 << 23) && p.ldb < (1 << 23));
  REQUIRE(p.lda >= (int64_t)p.chunks * 128 && p.ldb >= (int64_t)p.chunks * 128 && p.ldsa < (1 << 28) && p.ldsb < (1 << 28));
  REQUIRE(mode == MX_DENSE || (p.groups >= 1 && p.groups <= 256 && p.row_off));
  const __int128 tiles = (__int128)((p.m + 31) / 32 + (mode == MX_ROWS ? p.groups : 0)) * ((p.n + 31) / 32) * (mode == MX_K ? p.groups : 1);
  REQUIRE(tiles < ((__int128)1 << 31));
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_moe_plan(const int32_t*, int tokens, int topk, int64_t ldidx, int groups, int pad, int32_t*, int32_t*,
                           int32_t*, int cap, int32_t*, int32_t*, hipStream_t) {
  REQUIRE(tokens > 0 && topk > 0 && (int64_t)tokens * topk < (1 << 30) && ldidx >= topk && groups >= 1 && groups <= 256);
  REQUIRE(pad >= 1 && pad <= 1024 && cap >= tokens * topk + groups * (pad - 1));
  ++g_launches;
  return hipSuccess;
}
int64_t moe_balance_workspace(int64_t tokens, int64_t experts, int64_t sequences) { return tokens + experts + sequences; }
hipError_t launch_moe_balance(const MoeBalanceArgs& a, int, bool, float*, int32_t*, int32_t*, void*, hipStream_t) {
  REQUIRE(a.tokens > 0 && a.experts >= 1 && a.experts <= 1024 && a.sequences >= 1 && (a.seq_off || a.sequences == 1));
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_moe_balance_grad(const MoeBalanceArgs& a, int, bool, const float*, const int32_t*, const int32_t*, void*,
                                   int64_t lddl, hipStream_t) {
  REQUIRE(a.tokens > 0 && lddl >= a.experts);
  ++g_launches;
  return hipSuccess;
}
}  // namespace fp8bq

int main() {
  // every size argument of every entry point set to each of these, one at a time and two at a time
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 31, 256, 300, 1 << 20, (1ll << 28) - 1, 1ll << 31, 1ll << 40, INT64_MAX - 255, INT64_MAX};
  const int n = sizeof(sizes) / sizeof(sizes[0]);
  void* p = reinterpret_cast<void*>(0x10000);
  int32_t* i = reinterpret_cast<int32_t*>(0x20000);
  float* f = reinterpret_cast<float*>(0x30000);
  long calls = 0;
  auto sweep = [&](int count, const int64_t* good, auto&& call) {
    int64_t a[16];
    for (int x = 0; x < count; ++x)
      for (int y = x; y < count; ++y)
        for (int u = 0; u < n; ++u)
          for (int v = 0; v < n; ++v) {
            std::memcpy(a, good, sizeof(int64_t) * count);
            a[x] = sizes[u];
            a[y] = sizes[v];
            call(a);
            ++calls;
          }
  };
  const int64_t quant[] = {70, 300, 300, 256, 70, 128, 300};
  sweep(7, quant, [&](int64_t* a) {
    for (int t = 0; t < 4; ++t) fp8bq_quant_mxfp4_1x32(p, t, a[0], a[1], a[2], p, a[3], p, a[4], t & 1 ? nullptr : p, a[5], t & 1 ? nullptr : p, a[6], t & 1 ? 0x20 : 0, nullptr);
  });
  const int64_t disp[] = {20, 300, 300, 70, 256, 70, 128, 300};
  sweep(8, disp, [&](int64_t* a) {
    fp8bq_dispatch_mxfp4_1x32(p, 0, a[0], a[1], a[2], i, a[3], p, a[4], p, a[5], nullptr, a[6], nullptr, a[7], 0, p, nullptr);
  });
  const int64_t deq[] = {70, 300, 256, 70, 300};
  sweep(5, deq, [&](int64_t* a) { fp8bq_dequant_mxfp4_1x32(p, a[0], a[1], a[2], p, a[3], p, 2, a[4], nullptr); });
  const int64_t gemm[] = {70, 90, 300, 256, 70, 256, 90, 90, 4};
  sweep(9, gemm, [&](int64_t* a) {
    fp8bq_gemm_mxfp4(a[0], a[1], a[2], p, a[3], p, a[4], p, a[5], p, a[6], p, 2, a[7], nullptr);
    fp8bq_grouped_gemm_mxfp4((int32_t)a[8], i, a[0], a[1], a[2], p, a[3], p, a[4], p, a[5], p, a[6], p, 0, a[7], nullptr);
    fp8bq_grouped_wgrad_mxfp4((int32_t)a[8], i, a[0], a[1], a[2], p, a[3], p, a[4], p, a[5], p, a[6], p, 2, a[7], nullptr);
  });
  const int64_t plan[] = {100, 8, 8, 32, 1288, 16};
  sweep(6, plan, [&](int64_t* a) { fp8bq_moe_plan(i, a[0], a[1], a[2], (int32_t)a[5], a[3], i, i, i, a[4], i, p, nullptr); });
  const int64_t bal[] = {100, 64, 64, 6, 6, 3, 64};
  sweep(7, bal, [&](int64_t* a) {
    int64_t bytes;
    fp8bq_moe_balance_workspace_size(a[0], a[1], a[5], &bytes);
    fp8bq_moe_balance(p, 2, a[0], a[1], a[2], i, a[3], a[4], i, a[5], 0, 1.f, f, i, i, p, nullptr);
    fp8bq_moe_balance_grad(f, p, 0, a[0], a[1], a[2], i, a[3], a[4], nullptr, a[5], 1, 1.f, i, i, p, a[6], nullptr);
  });
  std::printf("%ld sweeps, %d accepted calls\n", calls, g_launches);
  return g_launches > 100 ? 0 : 1;
}
