// Which tiling an MXFP4 product runs on, from its sizes alone. Host only, free of
// HIP, so that a test can ask which kernel a size goes to.
#pragma once

#include <stdint.h>

namespace fp8bq {

enum MxMode { MX_DENSE = 0, MX_ROWS = 1, MX_K = 2 };   // one product; rows grouped; K grouped

// Which kernel. A product's time is close to rounds x (chunks x step + store)
// + launch, where a round is one tile on each of the 256 CUs (several
// workgroups of the small tilings share a CU; their steps then take turns).
// Step and store times in units of 10 ns, from products of 1 x 2048 x 7168 to
// 16384 x 18432 x 7168; a tile twice as large takes less than twice the step, as
// long as there are enough of them. Measured (us, bf16 out):
//                       stream   64x64  64x128 128x128 128x256 256x256
//   1 x 2048 x 7168        6.8    11.7    13.0    15.3    26.5    38.8
//   1 x 18432 x 7168      18.2    17.1    14.4    16.9    29.8    40.0
//   48 x 18432 x 7168     39.5    17.9    14.9    17.0    29.7    40.0
//   1000 x 4096 x 7168   114.5    32.7    28.6    21.2    31.1    42.4
//   2048 x 2048 x 2048    41.1    13.7    12.8     9.2    12.5    17.5
//   4096 x 2048 x 7168   226.9    62.0    52.8    38.3    35.6    45.1
//   4096 x 7168 x 2048   271.4    70.0    63.4    48.3    47.3    42.5
//   16384 x 18432 x 7168  9031    2102    1696    1227    1176     987
// (64 x 64, 64 x 128 and up to 256 tiles of 128 x 128 with loading waves.)
struct Tiling { int bm, bn, step, store; };
constexpr Tiling kTilings[] = {{32, 32, 25, 0}, {64, 64, 33, 40}, {64, 128, 42, 70}, {128, 128, 57, 130},
                               {128, 256, 100, 250}, {256, 256, 170, 500}};

// The tiling with the least estimated time for `groups` products of rows x n x
// chunks each (an expert's rows are taken as their average: only the device
// knows the counts).
inline int pick_tiling(int64_t groups, int64_t rows, int64_t n, int64_t chunks) {
  int best = 5;
  double least = 0;
  for (int i = 0; i < 6; ++i) {
    const Tiling& t = kTilings[i];
    const int64_t tiles = groups * ((rows + t.bm - 1) / t.bm) * ((n + t.bn - 1) / t.bn);
    const double time = (double)((tiles + 255) / 256) * (double)(chunks * t.step + t.store);
    if (i == 0 && tiles > 65536) continue;           // one workgroup per tile: keep the launch's thread count in range
    if (least == 0 || time < least) {
      best = i;
      least = time;
    }
  }
  return best;
}

// The tiling (its place in kTilings) of a product of m x n x chunks; deep: 128 x 128
// tiles with loading waves and a third stage.
struct MxPick { int tiling; bool deep; };
inline MxPick mx_pick(MxMode mode, int groups, int64_t m, int64_t n, int64_t chunks) {
  // Experts: their rows (or chunks of K) as the average of what the buffers
  // hold. Rows count half of that: a plan's buffer has room for every choice of
  // every token, many of which may be other GPUs' experts, and too large a tile
  // costs more than too small a one (8 experts with 57 .. 232 rows in a buffer
  // of 2048, n = 2048, k = 7168: 20.8 us with 64 x 128, 33.5 with 128 x 128
  // without loading waves). What the guess costs, n = 2048, k = 7168 (us, this
  // rule / the best tiling):
  //   8 of 256 experts, even:  512 of 16384 rows    44.7 / 20.3 (64 x 128)
  //                            2048 of 65536        50.4 / 25.9 (128 x 128, deep)
  //                            16384 of 524288       118 / 118
  //   8 of 8, even:            2048 of 2048         29.9 / 27.5 (128 x 128, deep)
  //                            16384 of 16384        118 / 118
  // and of 32 experts, n = 1024, k = 2048, 8192 of 65536 rows 25.5 / 17.7 (128 x
  // 256), 16384 of 16384 28.5 / 26.3 (256 x 256), 2048 of 2048 12.3 / 12.3.
  const int64_t g = mode == MX_DENSE ? 1 : groups;
  const int64_t rows = mode == MX_ROWS ? (m + 2 * g - 1) / (2 * g) : m;
  // one 128 x 128 tile per CU or less: loading waves and a third stage hide more
  // latency (1000 x 4096 x 7168: 22.5 against 25.9 us); with more, two workgroups
  // per CU do better (4096 x 2048 x 7168: 37.2 against 38.8)
  const bool deep = g * ((rows + 127) / 128) * ((n + 127) / 128) <= 256;
  return {pick_tiling(g, rows, n, mode == MX_K ? (chunks + g - 1) / g : chunks), deep};
}

}  // namespace fp8bq
