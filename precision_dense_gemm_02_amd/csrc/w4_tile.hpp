// Host side of the products with 4-bit weights: the kernel for the sizes and
// its launch.  run_w4_tile<T, STEPS> is instantiated in translation units of
// its own (run_w4_*.hip).
#pragma once

#include "../../include/lpgemm_ffn.h"
#include "dispatch.hpp"
#include "ffn.hpp"
#include "w4_tile_kernels.hpp"

namespace lpgemm {

enum W4Way {
  W4_FEW_ROWS = 0,   // few_rows
  W4_TILE = 1,       // w4_tile
  W4_WHOLE = 2,      // the weights as 16-bit values in the workspace, then the block's tiles
};
struct W4Plan {
  int way;
  int bm;            // W4_TILE: 32 or 64 rows by 128 columns
  int splits;
};

// Up to this many rows the weights enter the sums exactly; beyond, they are
// first written out as 16-bit values, each rounded once.  The tiles with exact
// weights against that, in us: 32 rows x 14336 x 4096 21 and 62; 256 rows x 4096 x 14336 63 and 91, x 14336 x 4096
// 76 and 94, gated x 14336 x 4096 129 and 140; 384 rows 102 and 103, 114 and 99,
// 192 and 166; 512 rows 114 and 129, 152 and 102, 237 and 162; 1024 rows 224 and
// 146, 272 and 143, 468 and 266.  (4096 x 4096: 384 rows 32 and 37, 512 34 and 38,
// 768 64 and 59, 2048 127 and 78.)
constexpr int kW4ExactRows = LPGEMM_W4_EXACT_M;

// N: weight rows (gated: both projections').  In us, few rows' kernel against the
// best tiles: 16 x 4096 x 4096 8.7 and 11.5, 16 x 14336 x 4096 18.6 and 19.9, but
// 16 x 28672 x 4096 30.1 and 22.8; 32 x 4096 x 4096 11.9 and 12.7, but 32 x 4096 x
// 14336 33.2 and 20.5.  Tiles against 16-bit weights: at kW4ExactRows.
inline W4Plan plan_w4(int64_t M, int64_t N, int64_t K, int cu_count) {
  const int64_t weights = N * K;
  W4Plan plan{W4_TILE, 32, 1};
  if (M > kW4ExactRows) plan.way = W4_WHOLE;
  else if (M <= LPGEMM_W4_SHORT_M || (M <= 16 && N < 20480) || weights <= (M <= 32 ? (int64_t)20 << 20 : M <= 64 ? (int64_t)8 << 20 : 0))
    plan.way = W4_FEW_ROWS;
  const int forced = forced_ffn();
  if (M > LPGEMM_W4_SHORT_M && forced >= FFN_FEW_ROWS && (forced != FFN_FEW_ROWS || M <= 16 * 65535)) plan.way = forced == FFN_FEW_ROWS ? W4_FEW_ROWS : forced == FFN_W4_WHOLE ? W4_WHOLE : W4_TILE;
  if (plan.way != W4_TILE) return plan;
  if ((int64_t)tiles(M, 32) * tiles(N, 128) > cu_count) plan.bm = 64;
  if (forced == FFN_W4_32) plan.bm = 32;
  if (forced == FFN_W4_64) plan.bm = 64;
  const int64_t n = (int64_t)tiles(M, plan.bm) * tiles(N, 128), stages = tiles(K, 128);
  int64_t s = cu_count / n;
  if (s > stages / 8) s = stages / 8;
  if (s > 16) s = 16;
  if (s > 1) plan.splits = (int)s;
  return plan;
}

inline int64_t w4_part_bytes(const W4Plan& p, int64_t M, int64_t N) { return p.way == W4_TILE && p.splits > 1 ? 4 * p.splits * M * N : 0; }

template <typename T, int STEPS>
lpgemm_status run_w4_tile(const W4Plan& plan, W4TileArgs p, hipStream_t stream);

#ifdef LPGEMM_W4_DEFINE
template <typename T, int STEPS, bool GATED>
const void* w4_kernel(int bm) {
  return bm == 32 ? (const void*)&w4_tile<T, STEPS, 32, 2, 4, GATED> : (const void*)&w4_tile<T, STEPS, 64, 2, 2, GATED>;
}

template <typename T, int STEPS>
lpgemm_status run_w4_tile(const W4Plan& plan, W4TileArgs p, hipStream_t stream) {
  p.stages = tiles(p.K, 128);
  p.split_stages = tiles(p.stages, plan.splits);
  p.splits = plan.splits;
  p.tiles_m = tiles(p.M, plan.bm);
  p.tiles_n = p.F > 0 ? tiles(p.F, 64) : tiles(p.N, 128);
  void* kargs[] = {&p};
  const void* fn = p.F > 0 ? w4_kernel<T, STEPS, true>(plan.bm) : w4_kernel<T, STEPS, false>(plan.bm);
  if (hipLaunchKernel(fn, dim3((unsigned)(p.tiles_m * p.tiles_n), (unsigned)plan.splits), dim3(plan.bm == 32 ? 1024 : 512), kargs, 0, stream) != hipSuccess)
    return LPGEMM_ERROR_LAUNCH;
  if (plan.splits == 1) return LPGEMM_SUCCESS;
  const int64_t n = (int64_t)p.M * (p.F > 0 ? p.F : p.N);
  return hipLaunchKernel((const void*)&join_w4<T>, dim3((unsigned)((n + 255) / 256)), dim3(256), kargs, 0, stream) == hipSuccess
             ? LPGEMM_SUCCESS
             : LPGEMM_ERROR_LAUNCH;
}
#endif

}  // namespace lpgemm
