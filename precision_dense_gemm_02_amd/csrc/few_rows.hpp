// Host side of the products of few rows: the kernel for the sizes and its
// launch.  run_few_rows<T> is instantiated once per type in its own
// translation unit (run_few_rows_*.hip).
#pragma once

#include "../../include/lpgemm_ffn.h"
#include "dispatch.hpp"
#include "few_rows_kernels.hpp"

namespace lpgemm {

// w4: 0 for 16-bit weights, 1, 2 and 4 for groups of 32, 64 and 128 or more.
template <typename T>
lpgemm_status run_few_rows(const FewRowsArgs& p, int w4, int cu_count, hipStream_t stream);

#ifdef LPGEMM_FEW_ROWS_DEFINE
template <typename T, int W4>
const void* few_rows_kernel(int mt, int nb) {
  if (mt == 1) return nb == 4 ? (const void*)&few_rows<T, W4, 1, 4> : nb == 2 ? (const void*)&few_rows<T, W4, 1, 2> : (const void*)&few_rows<T, W4, 1, 1>;
  if (mt == 2) return nb == 2 ? (const void*)&few_rows<T, W4, 2, 2> : (const void*)&few_rows<T, W4, 2, 1>;
  return nb == 2 ? (const void*)&few_rows<T, W4, 4, 2> : (const void*)&few_rows<T, W4, 4, 1>;
}

template <typename T>
lpgemm_status run_few_rows(const FewRowsArgs& args, int w4, int cu_count, hipStream_t stream) {
  FewRowsArgs p = args;
  const bool gated = p.F > 0;
  const int columns = gated ? p.F : p.N;
  const int mt = p.M <= 16 ? 1 : p.M <= 32 ? 2 : 4;
  auto grid = [&](int nb) { return tiles(columns, 16 * (gated ? nb / 2 : nb)); };
  int nb = gated ? 2 : 1;
  if (!gated && grid(2) >= cu_count) nb = 2;
  if (mt == 1 && grid(4) >= 2 * cu_count) nb = 4;
  const int blocks = (p.K + 127) / 128;
  int waves = few_rows_waves(mt, nb);
  if (grid(nb) > cu_count && waves > 8) waves = 8;
  while (waves > 1 && waves / 2 >= blocks) waves /= 2;
  const size_t lds = (size_t)waves * 16 * mt * (16 * nb + 1) * 4;
  const void* fn = w4 == 0 ? few_rows_kernel<T, 0>(mt, nb)
                 : w4 == 1 ? few_rows_kernel<T, 1>(mt, nb)
                 : w4 == 2 ? few_rows_kernel<T, 2>(mt, nb)
                           : few_rows_kernel<T, 4>(mt, nb);
  void* kargs[] = {&p};
  return hipLaunchKernel(fn, dim3((unsigned)grid(nb), (unsigned)tiles(p.M, 16 * mt)), dim3(64 * waves), kargs, lds,
                         stream) == hipSuccess
             ? LPGEMM_SUCCESS
             : LPGEMM_ERROR_LAUNCH;
}
#endif

}  // namespace lpgemm
