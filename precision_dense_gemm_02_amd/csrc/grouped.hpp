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
  GCFG_SKINNY_8 = 0,    // 8 rows x 32 columns, waves split K
  GCFG_SKINNY_16 = 1,
  GCFG_SKINNY_32 = 2,
  GCFG_64x128 = 3,
  GCFG_128x128 = 4,
  GCFG_256x256 = 5,
  GCFG_COUNT = 6
};

inline int grouped_tile_rows(int cfg) {
  switch (cfg) {
    case GCFG_SKINNY_8: return 8;
    case GCFG_SKINNY_16: return 16;
    case GCFG_SKINNY_32: return 32;
    case GCFG_64x128: return 64;
    case GCFG_128x128: return 128;
    default: return 256;
  }
}
inline int grouped_tile_cols(int cfg) {
  return cfg <= GCFG_SKINNY_32 ? 32 : (cfg <= GCFG_128x128 ? 128 : 256);
}

// The most row tiles of `tile` rows that `rows` rows in `groups` groups can
// make: every non-empty group may end in a partial tile.
inline int64_t grouped_max_tiles(int64_t rows, int64_t groups, int tile) {
  const int64_t used = groups < rows ? groups : rows;
  return (rows + used * (tile - 1)) / tile;
}

inline GroupedCfg choose_grouped(int64_t rows, int64_t groups, int64_t N, int cu_count) {
  const int64_t used = groups < rows ? groups : rows;
  const int64_t mean = (rows + used - 1) / used;
  if (mean <= 32) return rows <= 8 ? GCFG_SKINNY_8 : (rows <= 16 ? GCFG_SKINNY_16 : GCFG_SKINNY_32);
  if (mean <= 64) return GCFG_64x128;
  if (mean >= 192 && 2 * used * tiles(mean, 256) * tiles(N, 256) > cu_count) return GCFG_256x256;
  return GCFG_128x128;
}

template <int KIND>
lpgemm_status run_grouped(GroupedArgs p, int cu_count, hipStream_t stream);

#ifdef LPGEMM_GROUPED_DEFINE
template <int KIND>
lpgemm_status run_grouped(GroupedArgs p, int cu_count, hipStream_t stream) {
  const GroupedCfg cfg = choose_grouped(p.rows, p.groups, p.N, cu_count);
  p.k_stages = (p.row_bytes + 127) / 128;
  p.tiles_n = tiles(p.N, grouped_tile_cols(cfg));
  const int64_t grid = grouped_max_tiles(p.rows, p.groups, grouped_tile_rows(cfg)) * p.tiles_n;
  if (grid > INT32_MAX) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  const void* fn = nullptr;
  switch (cfg) {
    case GCFG_SKINNY_8: fn = (const void*)&grouped_skinny<KIND, 4, 4, 1>; break;
    case GCFG_SKINNY_16: fn = (const void*)&grouped_skinny<KIND, 4, 4, 2>; break;
    case GCFG_SKINNY_32: fn = (const void*)&grouped_skinny<KIND, 4, 4, 4>; break;
    case GCFG_64x128: fn = (const void*)&grouped_tile<KIND, 64, 128, 2, 2, 4, false>; break;
    case GCFG_128x128: fn = (const void*)&grouped_tile<KIND, 128, 128, 2, 2, 4, false>; break;
    default: fn = (const void*)&grouped_tile<KIND, 256, 256, 2, 2, 2, true>; break;
  }
  void* kargs[] = {&p};
  return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(256), kargs, 0, stream) == hipSuccess ? LPGEMM_SUCCESS
                                                                                             : LPGEMM_ERROR_LAUNCH;
}
#endif

}  // namespace lpgemm
