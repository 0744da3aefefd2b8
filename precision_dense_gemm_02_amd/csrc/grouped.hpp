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
// one).  Measured with every kernel at 2016 sizes: one group of 1 to 6000
// rows, and 4 to 128 groups of 1 to 600 rows each on average, evenly and
// unevenly spread, N = 512 to 14336, K = 1024 to 7168, with weights that are
// in no cache (graph replay, one MI355X).  At 756 other sizes the choice is 3%
// (int8), 2% (binary16, MXFP4 experts) and 1% (one group) behind the best
// kernel of each in the geometric mean, a tenth of them by 12, 9, 8 and 3% or
// more, the worst 1.6 times.  The figures at each rule are us of the kernel it
// takes against another, or of both where it turns.
inline GroupedCfg choose_grouped(int kind, int64_t rows, int64_t groups, int64_t N, int64_t row_bytes, int cu_count) {
  const int64_t used = groups < rows ? groups : rows;
  const int64_t mean = (rows + used - 1) / used;
  const bool one = used == 1, f16 = kind == KIND_F16, mxfp4 = kind == KIND_MXFP4;
  // workgroups of a configuration, and whether they reach `percent` of the CUs
  auto grid = [&](GroupedCfg c) {
    const int64_t ragged = rows / grouped_tile_rows(c) + (used + 1) / 2, most = (4 * used + 4) / 5;
    const int64_t t = one ? tiles(rows, grouped_tile_rows(c)) : ragged > most ? ragged : most;
    return t * tiles(N, grouped_tile_cols(c));
  };
  auto fills = [&](GroupedCfg c, int64_t percent) { return 100 * grid(c) >= percent * cu_count; };
  // percent of a round of `slots` workgroups; the first four rounds count whole
  auto rounds = [](int64_t t, int64_t slots) { return t <= 4 * slots ? 100 * ((t + slots - 1) / slots) : 100 * t / slots; };
  // MXFP4 experts with 100 MiB of weights and more, mostly read by one row
  // tile: B streams non-temporally.  A model's layers together hold more than
  // the 256 MiB Infinity Cache, so the weights are taken not to be in it when
  // the call comes.  Then the stream is faster at every size (us with and
  // without, 8 rows an expert: 64 experts of 2048 x 2048, 128 MiB, 29.5, 32.6;
  // 32 of 7168 x 2048, 224 MiB, 50.3, 53.7; 64 of 2048 x 4096, 256 MiB, 50.1,
  // 57.0; 128 of 4096 x 4096, 1 GiB, 193, 212).  A call that repeats on the
  // same weights pays below 256 MiB, as it finds less of them cached (29.0,
  // 26.5; 49.7, 43.7), and gains from there on (50.4, 51.6; 198, 219).  Below
  // 100 MiB the weights of two such calls fit in the cache together: plain
  // loads.  Rows that do not start on a cache line: 1.25 times slower, each
  // line is fetched twice.  K = 1024, four lines a row: no faster (64 of 7168 x
  // 1024 26.6 against 25.6).
  // (divided by the groups: the product of all three may pass 64 bits)
  const int64_t least = (((int64_t)100 << 20) + groups - 1) / groups;
  if (mxfp4 && !one && row_bytes % 128 == 0 && row_bytes > 512 && N * row_bytes >= least) {
    if (mean > 16 && mean < 96) return GCFG_128x128_NT;
    if (mean > 4 && mean <= 16) return GCFG_64x64_NT;
  }
  // few rows per group: the weights' stream is the work, and narrow tiles
  // whose waves split K keep most of it in flight.  One group up to 20 rows
  // (MXFP4 18 x 7168 x 4096: 6.4 against 8.9 on 64 x 64 tiles; 36 x 14336 x
  // 7168: 26.8 against 14.6).  Several, int8, up to 12 rows each (31 groups of
  // 12, 1416 x 4096: 34.4 against 43.6; of 15, 2048 x 1024: 23.2 against
  // 17.4); binary16, twice the bytes, up to 20 (31 groups of 19, 2048 x 2048:
  // 49.3 against 60.0; of 32, 7168 x 1024: 142 against 92); MXFP4, half the
  // bytes, up to 10, and where eight stages or fewer leave a wave two, only
  // while there are few workgroups (31 groups of 7, 7168 x 1024: 41.0 against
  // 33.2; one row, 2048 x 1024: 5.9 against 7.1)
  const int64_t limit = one || f16 ? 20 : mxfp4 ? 10 : 12;
  const bool shallow = mxfp4 && !one && row_bytes <= 1024 && fills(GCFG_64x64_S2, 150);
  if (mean > limit || shallow) {
    // 256 x 256 tiles, one workgroup on a CU, or 128 x 128, two: a round of the
    // former takes 1.6 rounds of the latter (MXFP4, 288 tiles in two rounds of
    // 256, 4357 x 4096 x 2048: 33.0 on 128 x 128 against 41.3; 176 in one,
    // 2697 x 4096 x 4096: 32.5 on 256 x 256 against 40.6; int8, 16 groups of
    // 350 rows, 2048 x 4096: 256 x 256 is 1.3 times faster)
    if ((one || mean >= 96) && 160 * rounds(grid(GCFG_256x256), cu_count) <= 100 * rounds(grid(GCFG_128x128), 2 * cu_count))
      return GCFG_256x256;
    // two workgroups of 128 x 128 tiles share a CU: one's stores and first
    // loads behind the other's products (MXFP4 1280 x 14336 x 4096: 60.3
    // against 80.1 on 64 x 128; int8, 16 groups of 143 rows, 2048 x 4096: 46.6
    // against 51.9; less than a tile per CU, MXFP4 677 x 4096 x 4096: 19.2
    // against 17.5)
    if (mean >= (one ? 48 : 32) && fills(GCFG_128x128, one ? 105 : 130)) return GCFG_128x128;
    // (MXFP4 788 x 4096 x 7168: 28.6 against 31.6 on 64 x 64 tiles; binary16,
    // whose stage holds half the k, keeps the deeper ring of 64 x 64 at few
    // rows: 64 groups of 24, 2048 x 2048: 111 against 140)
    if (mean >= (f16 ? 32 : 24) && fills(GCFG_64x128, 150)) return GCFG_64x128;
    // up to two tiles per CU: the deeper ring (MXFP4 181 x 7168 x 4096: 14.0
    // against 16.7); beyond that: more workgroups (677 x 4096 x 4096: 17.5
    // against 20.1)
    if (!f16 && fills(GCFG_64x64_S2, 201)) return GCFG_64x64_S2;
    if (fills(GCFG_64x64_S4, one || mean >= 48 ? 45 : 60)) return GCFG_64x64_S4;
  }
  // the lowest tile that keeps the workgroups near one per CU, up to what the
  // rows need (MXFP4 37 x 1024 x 4096: 8 rows 4.2, 32 rows 5.3; 45 x 4096 x
  // 4096: 32 rows 6.0, 8 rows 7.9); with several groups by their mean rows
  // (int8, 31 groups of 12, 1416 x 4096: 16 rows 34.4, 32 rows 36.6, 8 rows
  // 42.3; MXFP4, 64 of 1 or 2, 2048 x 4096: 8 rows 47.0, 16 rows 46.5).  Ring
  // of 2 blocks from two workgroups a CU on (MXFP4, 9 experts of one row, 2048
  // x 1024: 5.9 against 7.3 with 3; at K = 4096 10.0 against 9.5)
  if (mean <= (one ? 8 : f16 || mxfp4 ? 4 : 6) || !fills(GCFG_SKINNY_8, 101))
    return fills(GCFG_SKINNY_8, mxfp4 && !one ? 150 : 201) ? GCFG_SKINNY_8 : GCFG_SKINNY_8_DEEP;
  if (mean <= (one ? 16 : 12) || !fills(GCFG_SKINNY_16, 101)) return GCFG_SKINNY_16;
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
