// Host side of the block's products: the tile for the sizes and its launch.
// run_tile<T> is instantiated once per type in its own translation unit
// (run_ffn_*.hip).
#pragma once

#include "../../include/lpgemm_ffn.h"
#include "dispatch.hpp"
#include "ffn_kernels.hpp"

namespace lpgemm {

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

extern int g_tile_bm[5], g_tile_splits[5], g_few_limit;

// The tile and the splits of an M x N product over K (gated: N = 2 F).
inline TilePlan plan_tiles(int job, int64_t M, int64_t N, int64_t K, int cu_count) {
  auto count = [&](int bm, int bn) { return (int64_t)tiles(M, bm) * tiles(N, bn); };
  TilePlan plan{64, 128, 1};
  if (2 * count(256, 256) > cu_count && M > 128) plan = {256, 256, 1};
  else if (2 * count(128, 128) > cu_count && M > 64) plan = {128, 128, 1};
  if (g_tile_bm[job]) plan = {g_tile_bm[job], g_tile_bm[job] == 64 ? 128 : g_tile_bm[job], 1};
  const int64_t stages = tiles(K, 64), n = count(plan.bm, plan.bn);
  if (n > 0 && n * 2 <= cu_count) {
    int64_t s = cu_count / n;
    if (s > stages / 4) s = stages / 4;
    if (s > 16) s = 16;
    if (s > 1) plan.splits = (int)s;
  }
  if (g_tile_splits[job]) plan.splits = (int)(g_tile_splits[job] < stages ? g_tile_splits[job] : stages ? stages : 1);
  return plan;
}

// A row of a split's sums: chunks of eight columns (gated: both projections').
inline int64_t part_stride(int job, int64_t N) { return job == JOB_GATED ? 2 * ((N / 2 + 7) / 8 * 8) : (N + 7) / 8 * 8; }
inline int64_t split_bytes(const TilePlan& p, int job, int64_t M, int64_t N) {
  return p.splits > 1 ? 4 * p.splits * M * part_stride(job, N) : 0;
}

// Runs a product (its operands, sizes and outputs set in p) with the splits'
// sums in `part` where the plan has splits.
template <typename T>
lpgemm_status run_tile(int job, TileArgs p, float* part, int cu_count, hipStream_t stream);

#ifdef LPGEMM_FFN_DEFINE
template <typename T, bool A_ACROSS, bool B_ACROSS, int END>
const void* tile_kernel(const TilePlan& plan) {
  if (plan.bm == 256) return (const void*)&ffn_tile<T, A_ACROSS, B_ACROSS, 256, 256, 2, 2, 2, 3, END>;
  if (plan.bm == 128) return (const void*)&ffn_tile<T, A_ACROSS, B_ACROSS, 128, 128, 2, 2, 2, 3, END>;
  return (const void*)&ffn_tile<T, A_ACROSS, B_ACROSS, 64, 128, 2, 2, 3, 3, END>;
}

template <typename T>
lpgemm_status run_tile(int job, TileArgs p, float* part, int cu_count, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return LPGEMM_SUCCESS;
  const TilePlan plan = plan_tiles(job, p.M, p.N, p.K, cu_count);
  p.tiles_m = tiles(p.M, plan.bm);
  p.tiles_n = job == JOB_GATED ? tiles(p.F, plan.bn / 2) : tiles(p.N, plan.bn);
  p.k_stages = tiles(p.K, 64);
  p.split_stages = tiles(p.k_stages, plan.splits);
  p.splits = plan.splits;
  p.part = part;
  p.part_stride = (int)part_stride(job, p.N);
  const void *fn, *join;
  switch (job) {
    case JOB_GATED: fn = tile_kernel<T, false, false, END_GATED>(plan), join = (const void*)&join_splits<T, END_GATED>; break;
    case JOB_DOWN: fn = tile_kernel<T, false, false, END_STORE>(plan), join = (const void*)&join_splits<T, END_STORE>; break;
    case JOB_GATED_GRAD: fn = tile_kernel<T, false, true, END_GATED_GRAD>(plan), join = (const void*)&join_splits<T, END_GATED_GRAD>; break;
    case JOB_DX: fn = tile_kernel<T, false, true, END_STORE>(plan), join = (const void*)&join_splits<T, END_STORE>; break;
    default: fn = tile_kernel<T, true, true, END_STORE>(plan), join = (const void*)&join_splits<T, END_STORE>; break;
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
