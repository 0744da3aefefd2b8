// Host side of the block's products: the tile for the sizes and its launch.
// run_tile<T> is instantiated once per type in its own translation unit
// (run_ffn_*.hip), and for the products with 4-bit weights, whose sums are
// multiplied by factors, in two more (run_ffn_factors_*.hip).
#pragma once

#include "../../include/lpgemm_ffn.h"
#include "dispatch.hpp"
#include "ffn_kernels.hpp"

namespace lpgemm {

// What lpgemm_force_ffn_config pins.
enum FfnConfig {
  FFN_TILE_64 = 0,    // the block's products on 64 x 128 tiles
  FFN_TILE_128 = 1,   // ... 128 x 128
  FFN_TILE_256 = 2,   // ... 256 x 256
  FFN_FEW_ROWS = 3,   // few_rows: the block's forward pass, 4-bit weights
  FFN_W4_32 = 4,      // 4-bit weights: tiles of 32 rows
  FFN_W4_64 = 5,      // ... of 64 rows
  FFN_W4_WHOLE = 6,   // ... through 16-bit weights
  FFN_CONFIG_COUNT = 7
};
extern std::atomic<int> g_forced_ffn;   // (ffn.hip)
inline int forced_ffn() { return g_forced_ffn.load(std::memory_order_relaxed); }

// The products of the block.
enum TileJob {
  JOB_GATED = 0,       // [g u] = X . W_gate_up^T, with the activation
  JOB_DOWN = 1,        // y = h . W_down^T
  JOB_GATED_GRAD = 2,  // dh = dY . W_down, with the activation's gradient
  JOB_DX = 3,          // dX = [dg du] . W_gate_up
  JOB_DW = 4,          // dW = [dg du]^T . X, dY^T . h
};

struct TilePlan {
  int bm, bn;
  int splits;
};

// The tile and the splits of an M x N product over K (gated: N = 2 F): of the
// kernels' three tiles and up to 16 splits the pair whose time a model puts
// lowest.  The model, in us: the workgroups fill the CUs in rounds (two on a CU
// with tiles of 64 and 128 rows, one with 256); a round takes its stages, each
// longer the more workgroups share the chip, and a fixed time for its first
// loads and its end (which is longer where the end has an activation); splits
// add a launch and the traffic of their sums.  Its numbers were fitted to the
// times of every pair at 130 products (M, N and K of blocks of 16 to 4096 rows,
// D = 1024 to 4096, F = 1416 to 14336, one MI355X).  With the kernels as they are
// now the choice is 1.5% of the product's time behind the best pair on average,
// 22% at the worst (116 products; a new fit came to the same).
inline TilePlan plan_tiles(int job, int64_t M, int64_t N, int64_t K, int cu_count) {
  struct Tile {
    int bm, bn, per_cu;
    double stage, stage_full, ends;   // a stage with few workgroups and with all places taken, a workgroup's start and end
  };
  static constexpr Tile kTiles[] = {{64, 128, 2, 0.433, 0.96, 4.19}, {128, 128, 2, 0.527, 1.045, 7.51}, {256, 256, 1, 1.033, 1.33, 20.8}};
  const double end_factor = job == JOB_GATED_GRAD ? 1.71 : job == JOB_GATED ? 1.43 : 1.0;
  const double stages = (double)((K + 63) / 64);
  TilePlan best{64, 128, 1};
  double least = 1e300;
  const int forced = forced_ffn();
  for (const Tile& t : kTiles) {
    if (forced >= FFN_TILE_64 && forced <= FFN_TILE_256 && &t != &kTiles[forced]) continue;
    const double count = (double)((M + t.bm - 1) / t.bm) * (double)((N + t.bn - 1) / t.bn), places = (double)cu_count * t.per_cu;
    for (int splits = 1; splits <= 16 && (splits == 1 || 2 * splits <= stages); splits *= 2) {
      const double per_split = (double)(((int64_t)stages + splits - 1) / splits);
      auto round = [&](double workgroups) {
        const double shared = t.per_cu == 2 ? (workgroups - cu_count) / cu_count : (workgroups - cu_count / 4) / (0.75 * cu_count);
        const double share = shared < 0 ? 0 : shared > 1 ? 1 : shared;
        return workgroups > 0 ? per_split * (t.stage + (t.stage_full - t.stage) * share) + end_factor * t.ends : 0.0;
      };
      const double all = count * splits, full = (double)(int64_t)(all / places);
      // (many rounds: the workgroups no longer move together)
      double time = all > 4 * places ? (all / places + 0.3) * round(places) : full * round(places) + round(all - full * places);
      if (splits > 1) time += 6.19 + 0.355 * splits + (double)M * (double)N * (8.0 * splits + (job == JOB_GATED_GRAD ? 10 : 2)) / 10.0e6;
      if (time < least) least = time, best = {t.bm, t.bn, splits};
    }
  }
  return best;
}

// A row of a split's sums: chunks of eight columns (gated: both projections').
inline int64_t part_stride(int job, int64_t N) { return job == JOB_GATED ? 2 * ((N / 2 + 7) / 8 * 8) : (N + 7) / 8 * 8; }
inline int64_t split_bytes(const TilePlan& p, int job, int64_t M, int64_t N) {
  return p.splits > 1 ? 4 * p.splits * M * part_stride(job, N) : 0;
}

// Runs a product (its operands, sizes and outputs set in p) with the splits'
// sums in the `part_bytes` at `part` where the plan has splits.  (The plan is
// made again here: with another kernel pinned since the workspace was measured
// it may want more, and is refused.)
template <typename T, bool FACTORS = false>
lpgemm_status run_tile(int job, TileArgs p, float* part, int64_t part_bytes, int cu_count, hipStream_t stream);

#ifdef LPGEMM_FFN_DEFINE
template <typename T, bool A_ACROSS, bool B_ACROSS, int END, bool FACTORS>
const void* tile_kernel(const TilePlan& plan) {
  if (plan.bm == 256) return (const void*)&ffn_tile<T, A_ACROSS, B_ACROSS, 256, 256, 2, 2, 2, 3, END, FACTORS>;
  if (plan.bm == 128) return (const void*)&ffn_tile<T, A_ACROSS, B_ACROSS, 128, 128, 2, 2, 2, 3, END, FACTORS>;
  return (const void*)&ffn_tile<T, A_ACROSS, B_ACROSS, 64, 128, 2, 2, 3, 3, END, FACTORS>;
}

template <typename T, bool FACTORS>
lpgemm_status run_tile(int job, TileArgs p, float* part, int64_t part_bytes, int cu_count, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return LPGEMM_SUCCESS;
  const TilePlan plan = plan_tiles(job, p.M, p.N, p.K, cu_count);
  if (split_bytes(plan, job, p.M, p.N) > part_bytes) return LPGEMM_ERROR_INVALID_VALUE;
  p.tiles_m = tiles(p.M, plan.bm);
  p.tiles_n = job == JOB_GATED ? tiles(p.F, plan.bn / 2) : tiles(p.N, plan.bn);
  p.k_stages = tiles(p.K, 64);
  p.split_stages = tiles(p.k_stages, plan.splits);
  p.splits = plan.splits;
  p.part = part;
  p.part_stride = (int)part_stride(job, p.N);
  const void *fn, *join;
  auto take = [&](auto a_across, auto b_across, auto end) {
    fn = tile_kernel<T, decltype(a_across)::value, decltype(b_across)::value, decltype(end)::value, FACTORS>(plan);
    join = (const void*)&join_splits<T, decltype(end)::value, FACTORS>;
  };
  constexpr std::false_type along;
  constexpr std::integral_constant<int, END_STORE> store;
  if (job == JOB_GATED) take(along, along, std::integral_constant<int, END_GATED>());
  else if (FACTORS || job == JOB_DOWN) take(along, along, store);   // (4-bit weights lie along k)
  else if constexpr (!FACTORS) {
    constexpr std::true_type across;
    if (job == JOB_GATED_GRAD) take(along, across, std::integral_constant<int, END_GATED_GRAD>());
    else if (job == JOB_DX) take(along, across, store);
    else take(across, across, store);
  }
  void* kargs[] = {&p};
  if (hipLaunchKernel(fn, dim3((unsigned)(p.tiles_m * p.tiles_n), (unsigned)plan.splits), dim3(256), kargs, 0, stream) != hipSuccess)
    return LPGEMM_ERROR_LAUNCH;
  if (plan.splits == 1) return LPGEMM_SUCCESS;
  const int64_t chunks = (int64_t)p.M * (((job == JOB_GATED ? p.F : p.N) + 7) / 8);
  return hipLaunchKernel(join, dim3((unsigned)((chunks + 255) / 256)), dim3(256), kargs, 0, stream) == hipSuccess
             ? LPGEMM_SUCCESS
             : LPGEMM_ERROR_LAUNCH;
}
#endif

}  // namespace lpgemm
