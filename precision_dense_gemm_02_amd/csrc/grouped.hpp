// Host side of the grouped and MXFP4 products: the kernel for the sizes and
// its launch.  run_grouped<KIND> is defined here and instantiated once per
// kind in its own translation unit (run_grouped_*.hip).
#pragma once

#include "../../include/lpgemm_moe.h"
#include "dispatch.hpp"
#include "grouped_kernels.hpp"

namespace lpgemm {

// Kernels of the grouped products.
enum GroupedCfg {
  GCFG_SKINNY_8_DEEP = 0,  // 8 rows x 32 columns, waves split K, ring of 3 blocks
  GCFG_SKINNY_8 = 1,       // ... ring of 2 blocks (more workgroups per CU)
  GCFG_SKINNY_16 = 2,      // 16 rows
  GCFG_SKINNY_32 = 3,      // 32 rows
  GCFG_64x64_S4 = 4,       // 64 x 64 tiles, 4 stages
  GCFG_64x64_S2 = 5,       // ... 2 stages (more workgroups per CU)
  GCFG_64x128 = 6,
  GCFG_128x128 = 7,
  GCFG_256x256 = 8,
  GCFG_64x64_NT = 9,       // as 5 and 7, with B streamed non-temporally
  GCFG_128x128_NT = 10,    // (MXFP4; the other kinds run 5 and 7)
  GCFG_COUNT = 11
};

inline int grouped_tile_rows(int cfg) {
  constexpr int rows[GCFG_COUNT] = {8, 8, 16, 32, 64, 64, 64, 128, 256, 64, 128};
  return rows[cfg];
}
inline int grouped_tile_cols(int cfg) {
  constexpr int cols[GCFG_COUNT] = {32, 32, 32, 32, 64, 64, 128, 128, 256, 64, 128};
  return cols[cfg];
}

// The most row tiles of `tile` rows that `rows` rows in `groups` groups can
// make: every non-empty group may end in a partial tile.
inline int64_t grouped_max_tiles(int64_t rows, int64_t groups, int tile) {
  const int64_t used = groups < rows ? groups : rows;
  return (rows + used * (tile - 1)) / tile;
}

// The kernel for the sizes.  How the rows fall on the groups is known on the
// device only; the choice goes by the mean, and by how many tiles the rows
// would make if half the groups ended in a tile of their own (and most had
// one).  Measured at
// 250 sizes of one group (1 to 4096 rows) and of 8 to 128 groups (1 to 2048
// tokens, 2 or 8 experts each), N = 768 to 14336, K = 2048 to 14336 (graph
// replay, one MI355X; the figures at each rule are us with the kernel it
// takes against the next best).
inline GroupedCfg choose_grouped(int kind, int64_t rows, int64_t groups, int64_t N, int64_t row_bytes, int cu_count) {
  const int64_t used = groups < rows ? groups : rows;
  const int64_t mean = (rows + used - 1) / used;
  // tiles of a configuration, and whether they reach `percent` of the CUs
  auto fills = [&](GroupedCfg c, int64_t percent) {
    const int64_t ragged = rows / grouped_tile_rows(c) + (used + 1) / 2, most = (4 * used + 4) / 5;
    const int64_t t = used == 1 ? tiles(rows, grouped_tile_rows(c)) : ragged > most ? ragged : most;
    return 100 * t * tiles(N, grouped_tile_cols(c)) >= percent * cu_count;
  };
  // MXFP4 experts whose weights are more than the 256 MiB Infinity Cache keeps
  // from one call to the next, and mostly read by one row tile: B streams
  // non-temporally (64 experts of 2048 x 4096: 24 rows each 56.2 against 61.8
  // us, 12 rows 50.8 against 54.4; 128 of 1024 x 2048, 24 rows 35.4 against
  // 37.2; at 67 MB of weights 1.3-1.4 times slower, and with rows that do not
  // start on a cache line 1.25 times: each line is fetched twice)
  if (kind == KIND_MXFP4 && used > 1 && row_bytes % 128 == 0 && groups * N * row_bytes >= (int64_t)100 << 20) {
    if (mean > 16 && mean < 96) return GCFG_128x128_NT;
    if (mean > 4 && mean <= 16) return GCFG_64x64_NT;
  }
  // few rows per group: the weights' stream is the work, and narrow tiles
  // whose waves split K keep most of it in flight (int8, 8 tokens over 64
  // experts of 2048 x 2048: 22.9 against 25.4 us on 64 x 64 tiles; MXFP4,
  // 16 rows of 14336 x 4096: 8.9 against 10.3).  With several groups up to 12
  // rows each (64 groups of 16 rows: int8 51.7 on 64 x 64 tiles against 65.7);
  // MXFP4, half the bytes per row, up to 6 (8 rows: 31.4 against 34.8);
  // binary16, twice as many, up to 16 (16 rows: 103 against 104 and more).
  const bool few = used == 1 ? mean <= 16 : mean <= (kind == KIND_MXFP4 ? 6 : kind == KIND_F16 ? 16 : 12);
  if (!few) {
    // 256 x 256 tiles move the fewest bytes per product, but leave a ragged
    // group's last tile emptier (MXFP4 4096 x 4096 x 4096: 46.5 us against
    // 53.5 on 128 x 128; 8 groups of 512 rows, N = 14336: 227 against 231, at
    // N = 4096 59.5 against 44.4)
    if (used == 1 ? fills(GCFG_256x256, 60) : mean >= 256 && fills(GCFG_256x256, 250)) return GCFG_256x256;
    // two workgroups of 128 x 128 tiles share a CU: one's stores and first
    // loads behind the other's products (MXFP4 2048 x 4096 x 4096 28.1 against
    // 34.8 on 64 x 128; 3000 x 1536 x 3584 18.7 against 25.5; 1024 x 4096 x
    // 4096, one tile per CU, 20.6 against 19.4)
    if (mean >= 48 && fills(GCFG_128x128, 105)) return GCFG_128x128;
    // int8, 64 groups of 64 rows: 73.9 against 79.1 on 128 x 128 tiles; MXFP4
    // 256 x 14336 x 4096: 19.2 against 20.1; binary16, whose stage holds half
    // the k, keeps the deeper ring below 96 rows (64 groups of 25 rows, N =
    // 1500: 87.9 against 110)
    const bool f16 = kind == KIND_F16;
    if (mean >= (f16 ? 96 : 24) && fills(GCFG_64x128, 150)) return GCFG_64x128;
    // up to two tiles per CU: the deeper ring (MXFP4 512 x 4096 x 14336 34.1
    // against 37.9); beyond that: more workgroups (8 groups of 64 rows, N =
    // 4096: 12.9 against 16.3)
    if (!f16 && fills(GCFG_64x64_S2, 201)) return GCFG_64x64_S2;
    if (fills(GCFG_64x64_S4, 60)) return GCFG_64x64_S4;
  }
  // the lowest tile that keeps the workgroups near one per CU, up to what the
  // rows need (MXFP4 16 x 4096 x 4096: 8 rows 5.2 us, 16 rows 6.0; 32 rows
  // there: 8 rows 6.6, 16 rows 5.9; 64 rows: 32 rows 6.6, 16 rows 7.4)
  if (used == 1 ? mean <= 8 || !fills(GCFG_SKINNY_8, 126) : mean <= (kind == KIND_F16 ? 2 : 4))
    return fills(GCFG_SKINNY_8, 201) ? GCFG_SKINNY_8 : GCFG_SKINNY_8_DEEP;
  if (used == 1 ? mean <= 16 || !fills(GCFG_SKINNY_16, 126) : mean <= (kind == KIND_F16 ? 8 : 12))
    return GCFG_SKINNY_16;
  return GCFG_SKINNY_32;
}

// Columns per workgroup of the narrow kernels: of 32, 28, 24 and 16 the width
// that leaves the busiest CU the fewest columns, for t row tiles (N = 14336 in
// one row tile: 512 workgroups of 28 columns, two per CU, instead of 448 of
// 32: MXFP4 16 rows 8.4 against 8.7 us; N = 4096: 256 of 16 instead of 128,
// 4.8 against 5.1).  The wider on equal terms: every workgroup reads its rows
// of A.
inline int grouped_columns(int64_t t, int64_t N, int cu_count) {
  int best = 32;
  int64_t least = INT64_MAX;
  for (int w : {32, 28, 24, 16}) {
    const int64_t load = (t * tiles(N, w) + cu_count - 1) / cu_count * w;
    if (load < least) {
      least = load;
      best = w;
    }
  }
  return best;
}

// The kernel pinned by lpgemm_force_grouped_config, -1 for the choice above
// (grouped.hip).
extern std::atomic<int> g_forced_grouped;

template <int KIND>
lpgemm_status run_grouped(GroupedArgs p, int cu_count, hipStream_t stream);

#ifdef LPGEMM_GROUPED_DEFINE
template <int KIND>
lpgemm_status run_grouped(GroupedArgs p, int cu_count, hipStream_t stream) {
  const int forced = g_forced_grouped.load(std::memory_order_relaxed);
  GroupedCfg cfg = forced >= 0 ? (GroupedCfg)forced : choose_grouped(KIND, p.rows, p.groups, p.N, p.row_bytes, cu_count);
  if (KIND != KIND_MXFP4 && cfg == GCFG_64x64_NT) cfg = GCFG_64x64_S2;
  if (KIND != KIND_MXFP4 && cfg == GCFG_128x128_NT) cfg = GCFG_128x128;
  if (KIND == KIND_F16 && cfg == GCFG_64x64_S2) cfg = GCFG_64x64_S4;   // binary16 has the deeper ring only
  p.k_stages = (p.row_bytes + 127) / 128;
  p.tile_w = grouped_tile_cols(cfg);
  // (where the number of row tiles is known: one group, or about one row per
  // expert of a token)
  if (cfg <= GCFG_SKINNY_32 && (p.groups == 1 || p.rows <= 8))
    p.tile_w = grouped_columns(p.groups == 1 ? tiles(p.rows, grouped_tile_rows(cfg)) : p.rows, p.N, cu_count);
  p.tiles_n = tiles(p.N, p.tile_w);
  const int64_t grid = grouped_max_tiles(p.rows, p.groups, grouped_tile_rows(cfg)) * p.tiles_n;
  if (grid * 256 > UINT32_MAX) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;   // threads of one launch
  const void* fn = nullptr;
  switch (cfg) {
    case GCFG_SKINNY_8_DEEP: fn = (const void*)&grouped_skinny<KIND, 4, 3, 1>; break;
    case GCFG_SKINNY_8: fn = (const void*)&grouped_skinny<KIND, 4, 2, 1>; break;
    case GCFG_SKINNY_16: fn = (const void*)&grouped_skinny<KIND, 4, 2, 2>; break;
    case GCFG_SKINNY_32: fn = (const void*)&grouped_skinny<KIND, 4, 2, 4>; break;
    case GCFG_64x64_S4: fn = (const void*)&grouped_tile<KIND, 64, 64, 2, 2, 4, false, false>; break;
    case GCFG_64x64_S2:
      if constexpr (KIND != KIND_F16) fn = (const void*)&grouped_tile<KIND, 64, 64, 2, 2, 2, false, false>;
      break;
    case GCFG_64x64_NT:
      if constexpr (KIND == KIND_MXFP4) fn = (const void*)&grouped_tile<KIND, 64, 64, 2, 2, 2, false, false, true>;
      break;
    case GCFG_128x128_NT:
      if constexpr (KIND == KIND_MXFP4) fn = (const void*)&grouped_tile<KIND, 128, 128, 2, 2, 2, false, true, true>;
      break;
    case GCFG_64x128: fn = (const void*)&grouped_tile<KIND, 64, 128, 1, 4, 2, false, false>; break;
    case GCFG_128x128: fn = (const void*)&grouped_tile<KIND, 128, 128, 2, 2, 2, false, true>; break;
    default: fn = (const void*)&grouped_tile<KIND, 256, 256, 2, 2, 2, true, true>; break;
  }
  void* kargs[] = {&p};
  return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(256), kargs, 0, stream) == hipSuccess ? LPGEMM_SUCCESS
                                                                                             : LPGEMM_ERROR_LAUNCH;
}
#endif

}  // namespace lpgemm
