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
// The most wavefronts of a workgroup, and the blocks a wavefront has in flight:
// as many as the registers hold (128 of them for 16 wavefronts, 256 for 8).
constexpr int few_rows_waves(int mt, int nb) { return mt * nb == 1 ? 16 : 8; }
constexpr int few_rows_depth(int w4, int mt, int nb, bool x_lds, int waves) {
  if (x_lds) return w4 ? (nb == 1 ? 4 : 2) : nb == 2 ? 3 : 4;
  if (mt == 2) return w4 ? 1 : 2;
  if (waves == 16) return w4 ? 1 : 3;
  return nb == 1 ? 3 : nb == 2 ? 2 : 1;
}
template <typename T, int W4, bool ZEROS, int MT, int NB, bool XLDS, int WAVES>
const void* few_rows_of() {
  return (const void*)&few_rows<T, W4, ZEROS, MT, NB, XLDS, WAVES, few_rows_depth(W4, MT, NB, XLDS, WAVES)>;
}
template <typename T, int W4, bool ZEROS, int MT, bool XLDS>
const void* few_rows_kernel(int nb, int waves) {
  if constexpr (MT == 1 && !XLDS) {
    if constexpr (W4 != 0)
      if (nb == 4) return few_rows_of<T, W4, ZEROS, MT, 4, XLDS, 8>();
    if (nb == 1 && waves > 8) return few_rows_of<T, W4, ZEROS, MT, 1, XLDS, 16>();
  }
  return nb == 2 ? few_rows_of<T, W4, ZEROS, MT, 2, XLDS, 8>() : few_rows_of<T, W4, ZEROS, MT, 1, XLDS, 8>();
}
template <typename T, int W4, bool ZEROS>
const void* few_rows_kernel(int mt, int nb, int waves, bool x_lds) {
  return mt == 2 ? few_rows_kernel<T, W4, ZEROS, 2, false>(nb, waves)
         : x_lds ? few_rows_kernel<T, W4, ZEROS, 1, true>(nb, waves)
                 : few_rows_kernel<T, W4, ZEROS, 1, false>(nb, waves);
}

template <typename T>
lpgemm_status run_few_rows(const FewRowsArgs& args, int w4, int cu_count, hipStream_t stream) {
  FewRowsArgs p = args;
  const bool gated = p.F > 0;
  const int columns = gated ? p.F : p.N;
  const int mt = p.M <= 16 ? 1 : 2;
  auto grid = [&](int nb) { return tiles(columns, 16 * (gated ? nb / 2 : nb)); };
  const int blocks = (p.K + 127) / 128;
  p.x_lds_stride = blocks * 256 + 16;
  const int64_t x_lds = (int64_t)p.M * p.x_lds_stride;
  const bool in_lds = p.M <= 4 && x_lds <= 64 * 1024;
  // Column tiles a workgroup takes, and its waves.  With more workgroups than CUs
  // smaller ones fill them evenly; 4-bit weights then take four tiles, over which
  // an X fragment's loads and its sum are shared (bf16, 16 x 14336 x 4096, groups
  // of 64 with zeros: 16.9 us).
  int nb = gated ? 2 : 1, waves = 8;
  const bool many = grid(nb) > cu_count;
  if (in_lds) {
    if (many) waves = 4;
  } else if (mt == 1) {
    if (many && w4) nb = 4, waves = gated ? 4 : 8;
    else if (many) waves = 4;
    else waves = gated ? 8 : 16;
  } else {
    if (many) nb = 2, waves = 4;
    else if (w4 && tiles(p.M, 32) > 1) nb = 2;
  }
  if (waves > few_rows_waves(mt, nb)) waves = few_rows_waves(mt, nb);
  while (waves > 1 && waves / 2 >= blocks) waves /= 2;
  size_t lds = (size_t)waves * 16 * mt * (16 * nb + 1) * 4;
  if (in_lds && (size_t)x_lds > lds) lds = (size_t)x_lds;
  auto kernel = [&](auto w4_c) {
    constexpr int W4 = decltype(w4_c)::value;
    if constexpr (W4 != 0)
      if (p.zeros) return few_rows_kernel<T, W4, true>(mt, nb, waves, in_lds);
    return few_rows_kernel<T, W4, false>(mt, nb, waves, in_lds);
  };
  const void* fn = w4 == 0   ? kernel(std::integral_constant<int, 0>())
                   : w4 == 1 ? kernel(std::integral_constant<int, 1>())
                   : w4 == 2 ? kernel(std::integral_constant<int, 2>())
                             : kernel(std::integral_constant<int, 4>());
  void* kargs[] = {&p};
  return hipLaunchKernel(fn, dim3((unsigned)grid(nb), (unsigned)tiles(p.M, 16 * mt)), dim3(64 * waves), kargs, lds,
                         stream) == hipSuccess
             ? LPGEMM_SUCCESS
             : LPGEMM_ERROR_LAUNCH;
}
#endif

}  // namespace lpgemm
