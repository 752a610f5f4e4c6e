// Host-only driver for the entry points of the operators around a layer's
// Linears (csrc/api_layer.cpp with csrc/api.cpp), built with AddressSanitizer
// and UndefinedBehaviorSanitizer (g++, no GPU code): refusals with sizes up to
// INT64_MAX, and accepted calls through to stand-ins for the launchers that
// check what reaches them. Built and run by tests/test_abi_layer_sanitized.py.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "fp8bq.h"
#include "internal.h"
#include "layer.h"

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
// the last element of `rows` rows of `ld`, in bytes, fits 63 bits
bool reachable(int64_t rows, int64_t ld, int64_t bytes) { return (__int128)rows * ld * bytes <= INT64_MAX; }

hipError_t launch_rmsnorm(const NormArgs& a, int xtype, bool, hipStream_t) {
  REQUIRE(a.rows > 0 && a.rows < (1ll << 31) && a.cols > 0 && a.cols <= kNormMaxCols && xtype >= 0 && xtype <= 2 && a.wtype >= 0 && a.wtype <= 2);
  REQUIRE(a.x && a.w && (a.q || a.y) && !a.r == !a.h && !a.q == !a.s && a.eps >= 0);
  REQUIRE(a.ldx >= a.cols && reachable(a.rows, a.ldx, 4));
  REQUIRE(!a.r || (a.ldr >= a.cols && a.ldh >= a.cols && reachable(a.rows, a.ldr, 4) && reachable(a.rows, a.ldh, 4)));
  REQUIRE(!a.y || (a.ldy >= a.cols && reachable(a.rows, a.ldy, 4)));
  REQUIRE(!a.q || (a.cols % 128 == 0 && a.ldq >= a.cols && a.ldq % 16 == 0 && a.lds >= a.rows && reachable(a.cols / 128, a.lds, 4) && reachable(a.rows, a.ldq, 1)));
  ++g_launches;
  return hipSuccess;
}
int64_t norm_grad_parts(int64_t rows, int64_t) { return rows < 4096 ? rows : 4096; }
hipError_t launch_rmsnorm_grad(const NormGradArgs& a, int, hipStream_t) {
  REQUIRE(a.rows > 0 && a.rows < (1ll << 31) && a.cols > 0 && a.cols <= kNormMaxCols && a.dy && a.h && a.w && a.rstd && a.dx && a.dw && a.parts);
  REQUIRE(a.lddy >= a.cols && a.ldh >= a.cols && a.lddx >= a.cols && (!a.dh || (a.lddh >= a.cols && reachable(a.rows, a.lddh, 4))));
  REQUIRE(reachable(a.rows, a.lddy, 4) && reachable(a.rows, a.ldh, 4) && reachable(a.rows, a.lddx, 4));
  ++g_launches;
  return hipSuccess;
}
bool plan(int64_t tokens, int64_t rows, int64_t cols, int64_t topk) {
  return tokens > 0 && topk > 0 && rows > 0 && cols > 0 && (__int128)tokens * topk < (1 << 30) && rows < (1 << 30) && cols < (1ll << 31);
}
hipError_t launch_moe_dispatch(const MoeDispatchArgs& a, hipStream_t) {
  REQUIRE(plan(a.tokens, a.rows, a.cols, a.topk) && a.ldx >= a.cols && a.ldo >= a.cols && a.x && a.out && a.pos && a.src);
  REQUIRE(reachable(a.tokens, a.ldx, a.elem) && reachable(a.rows, a.ldo, a.elem) && (a.elem == 1 || a.elem == 2 || a.elem == 4));
  REQUIRE(!a.s == !a.so && (!a.s || (a.elem == 1 && a.cols % 128 == 0 && a.lds >= a.tokens && a.ldso >= a.rows &&
                                      reachable(a.cols / 128, a.lds, 4) && reachable(a.cols / 128, a.ldso, 4))));
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_moe_combine(const MoeCombineArgs& a, int, hipStream_t) {
  REQUIRE(plan(a.tokens, a.rows, a.cols, a.topk) && a.ldy >= a.cols && a.ldo >= a.cols && a.y && a.out && a.pos);
  REQUIRE(reachable(a.rows, a.ldy, 4) && reachable(a.tokens, a.ldo, 4) && (!a.w || (a.ldw >= a.topk && reachable(a.tokens, a.ldw, 4))));
  REQUIRE(!a.base || (a.ldb >= a.cols && reachable(a.tokens, a.ldb, 4)));
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_moe_combine_grad(const MoeCombineGradArgs& a, int, hipStream_t) {
  REQUIRE(plan(a.tokens, a.rows, a.cols, a.topk) && a.ldy >= a.cols && a.lddy >= a.cols && a.lddo >= a.cols && a.ldw >= a.topk);
  REQUIRE(a.dout && a.y && a.dy && a.w && a.dw && a.src && a.pos && reachable(a.rows, a.ldy, 4) && reachable(a.rows, a.lddy, 4));
  REQUIRE(reachable(a.tokens, a.lddo, 4) && reachable(a.tokens, a.ldw, 4));
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_gemv_mxfp4(const GemvArgs& p, int xtype, hipStream_t) {
  REQUIRE(p.m > 0 && p.n > 0 && p.k > 0 && p.xrows > 0 && p.x && p.b && p.sb && p.out && xtype >= 0 && xtype <= 2 && p.otype >= 0 && p.otype <= 2);
  REQUIRE(p.ldx >= p.k && p.ldo >= p.n && p.ldb >= (p.k + 255) / 256 * 128 && p.ldsb >= p.n && p.ldb % 16 == 0);
  REQUIRE(p.groups >= 0 && p.groups <= 256 && !p.groups == !p.row_off && (p.src || p.xrows >= p.m) && (p.m + 15) / 16 <= 65535);
  const int64_t tiles = (p.n + 15) / 16 * (p.groups ? p.groups : (p.m + 15) / 16);
  REQUIRE(tiles <= (1 << 23) && reachable(p.xrows, p.ldx, 4) && reachable(p.m, p.ldo, 4));     // of up to 512 threads: below 2^32
  REQUIRE(reachable(p.n, p.ldb, p.groups ? p.groups : 1) && reachable((p.k + 255) / 256 * 8, p.ldsb, p.groups ? p.groups : 1));
  ++g_launches;
  return hipSuccess;
}
}  // namespace fp8bq

int main() {
  // every size argument of every entry point set to each of these, one at a time and two at a time
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 31, 128, 256, 300, 1 << 20, (1ll << 28) - 1, 1ll << 31, 1ll << 40, INT64_MAX - 255, INT64_MAX};
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
  const int64_t norm[] = {70, 256, 256, 256, 256, 256, 256, 70};
  sweep(8, norm, [&](int64_t* a) {
    int64_t bytes;
    fp8bq_rmsnorm(p, 0, a[0], a[1], a[2], p, a[3], p, 2, 1e-6f, p, a[4], p, a[5], p, a[6], f, a[7], f, 0, nullptr);
    fp8bq_rmsnorm(p, 2, a[0], a[1], a[2], nullptr, a[3], p, 1, 0.f, nullptr, a[4], p, a[5], nullptr, a[6], nullptr, a[7], nullptr, 0x10, nullptr);
    fp8bq_rmsnorm_grad(p, 1, a[0], a[1], a[2], p, a[3], p, 0, f, a[7] & 1 ? nullptr : p, a[4], p, a[5], f, p, nullptr);
    if (fp8bq_rmsnorm_grad_workspace_size(a[0], a[1], &bytes) == 0 && bytes <= 0) std::abort();
  });
  const int64_t disp[] = {50, 256, 256, 50, 4, 300, 256, 300};
  sweep(8, disp, [&](int64_t* a) {
    fp8bq_moe_dispatch(p, 1, a[0], a[1], a[2], f, a[3], i, a[4], i, a[5], p, a[6], f, a[7], nullptr);
    for (int e = 0; e < 5; ++e) fp8bq_moe_dispatch(p, e, a[0], a[1], a[2], nullptr, a[3], i, a[4], i, a[5], p, a[6], nullptr, a[7], nullptr);
  });
  const int64_t comb[] = {300, 256, 256, 50, 4, 4, 256, 256};
  sweep(8, comb, [&](int64_t* a) {
    fp8bq_moe_combine(p, 2, a[0], a[1], a[2], i, a[3], a[4], f, a[5], p, a[6], p, a[7], nullptr);
    fp8bq_moe_combine(p, 0, a[0], a[1], a[2], i, a[3], a[4], nullptr, a[5], nullptr, a[6], p, a[7], nullptr);
    fp8bq_moe_combine_grad(p, 1, a[3], a[1], a[6], p, a[0], a[2], i, a[4], f, a[5], i, p, a[7], f, nullptr);
  });
  const int64_t gemv[] = {7, 90, 300, 300, 256, 90, 90, 20, 4};
  sweep(9, gemv, [&](int64_t* a) {
    fp8bq_gemv_mxfp4(a[0], a[1], a[2], p, 0, a[3], p, a[4], p, a[5], p, 2, a[6], nullptr);
    fp8bq_grouped_gemv_mxfp4((int32_t)a[8], i, a[0], a[1], a[2], p, 1, a[7], a[3], i, p, a[4], p, a[5], p, 1, a[6], nullptr);
    fp8bq_grouped_gemv_mxfp4((int32_t)a[8], i, a[0], a[1], a[2], p, 2, a[7], a[3], nullptr, p, a[4], p, a[5], p, 0, a[6], nullptr);
  });
  std::printf("%ld sweeps, %d accepted calls\n", calls, g_launches);
  return g_launches > 100 ? 0 : 1;
}
