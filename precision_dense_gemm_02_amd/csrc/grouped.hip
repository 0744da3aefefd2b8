// C entry points of the grouped products and of the MXFP4 product
// (include/lpgemm_moe.h).
#include "grouped.hpp"

namespace lpgemm {
std::atomic<int> g_forced_grouped{-1};
}  // namespace lpgemm

using namespace lpgemm;

namespace {

bool c_type(lpgemm_type t) { return t == LPGEMM_F32 || t == LPGEMM_F16 || t == LPGEMM_BF16; }

// The checks all kinds share, in the header's order.  `scales` tells whether
// the two scale pointers belong to the kind, `scale_align` what they need.
lpgemm_status check(int64_t rows, int64_t groups, int64_t N, int64_t K, int64_t a_rows, int64_t k_by, int64_t k_max,
                    int64_t row_bytes, const void* A, const void* B, bool grouped, const void* offsets,
                    const void* row_index, bool scales, const void* s0, const void* s1, int scale_align,
                    lpgemm_type type, const void* C, bool& nothing) {
  nothing = false;
  if (rows < 0 || groups < 0 || N < 0 || K < 0 || a_rows < 0) return LPGEMM_ERROR_INVALID_VALUE;
  if (rows > INT32_MAX || N > INT32_MAX || a_rows > INT32_MAX || !c_type(type)) return LPGEMM_ERROR_INVALID_VALUE;
  if (rows > 0 && !row_index && a_rows != rows) return LPGEMM_ERROR_INVALID_VALUE;
  if (K % k_by != 0 || K > k_max || groups > LPGEMM_MAX_GROUPS) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  // (a tile's last row and column must not leave 32 bits)
  if (rows > INT32_MAX - 256 || N > INT32_MAX - 256) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  if (row_index && a_rows * row_bytes >= ((int64_t)1 << 31)) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  if (rows == 0 || groups == 0 || N == 0) {
    nothing = true;
    return LPGEMM_SUCCESS;
  }
  const bool reads = K > 0 && a_rows > 0;
  if (!C || (grouped && !offsets) || (K > 0 && !B) || (reads && !A)) return LPGEMM_ERROR_INVALID_VALUE;
  if (scales && ((reads && !s0) || (K > 0 && !s1))) return LPGEMM_ERROR_INVALID_VALUE;
  if (!aligned16(C) || !aligned4(offsets) || !aligned4(row_index)) return LPGEMM_ERROR_MISALIGNED;
  if (K > 0 && (!aligned16(A) || !aligned16(B))) return LPGEMM_ERROR_MISALIGNED;
  const uintptr_t low = (uintptr_t)scale_align - 1;
  if (scales && ((reinterpret_cast<uintptr_t>(s0) & low) != 0 || (reinterpret_cast<uintptr_t>(s1) & low) != 0))
    return LPGEMM_ERROR_MISALIGNED;
  return LPGEMM_SUCCESS;
}

GroupedArgs args_of(int64_t rows, int64_t groups, int64_t N, int64_t a_rows, int64_t row_bytes, const void* A,
                    const void* B, const int32_t* offsets, const int32_t* row_index, lpgemm_type type, void* C) {
  GroupedArgs p{};
  p.A = static_cast<const uint8_t*>(A);
  p.B = static_cast<const uint8_t*>(B);
  p.offsets = offsets;
  p.row_index = row_index;
  p.C = static_cast<uint8_t*>(C);
  p.out_type = type;
  p.rows = (int)rows;
  p.a_rows = (int)a_rows;
  p.groups = (int)groups;
  p.N = (int)N;
  p.row_bytes = (int)row_bytes;
  return p;
}

lpgemm_status mxfp4(int64_t rows, int64_t groups, int64_t N, int64_t K, int64_t a_rows, const uint8_t* A,
                    const uint8_t* A_scale, const uint8_t* B, const uint8_t* B_scale, bool grouped,
                    const int32_t* offsets, const int32_t* row_index, lpgemm_type type, void* C, hipStream_t stream) {
  bool nothing;
  lpgemm_status st = check(rows, groups, N, K, a_rows, 32, LPGEMM_MAX_K_MXFP4, K / 2, A, B, grouped, offsets,
                           row_index, true, A_scale, B_scale, 16, type, C, nothing);
  if (st != LPGEMM_SUCCESS || nothing) return st;
  DeviceInfo dev;
  st = current_device(dev);
  if (st != LPGEMM_SUCCESS) return st;
  GroupedArgs p = args_of(rows, groups, N, a_rows, K / 2, A, B, offsets, row_index, type, C);
  p.a_scale = A_scale;
  p.b_scale = B_scale;
  p.scale_stride = (int)LPGEMM_MXFP4_SCALE_STRIDE(K);
  return run_grouped<KIND_MXFP4>(p, dev.cu_count, stream);
}

}  // namespace

extern "C" {

lpgemm_status lpgemm_i8_dequant_grouped(int64_t rows, int64_t groups, int64_t N, int64_t K, int64_t a_rows,
                                        const int8_t* A, const int8_t* B, const int32_t* offsets,
                                        const int32_t* row_index, const float* row_scale, const float* col_scale,
                                        lpgemm_type type, void* C, hipStream_t stream) {
  bool nothing;
  lpgemm_status st = check(rows, groups, N, K, a_rows, 16, LPGEMM_MAX_K_INT, K, A, B, true, offsets, row_index, true,
                           row_scale, col_scale, 4, type, C, nothing);
  if (st != LPGEMM_SUCCESS || nothing) return st;
  // the epilogue multiplies by the scales also where K = 0
  if ((a_rows > 0 && !row_scale) || !col_scale) return LPGEMM_ERROR_INVALID_VALUE;
  DeviceInfo dev;
  st = current_device(dev);
  if (st != LPGEMM_SUCCESS) return st;
  GroupedArgs p = args_of(rows, groups, N, a_rows, K, A, B, offsets, row_index, type, C);
  p.row_scale = row_scale;
  p.col_scale = col_scale;
  return run_grouped<KIND_I8_DEQUANT>(p, dev.cu_count, stream);
}

lpgemm_status lpgemm_f16_grouped(int64_t rows, int64_t groups, int64_t N, int64_t K, int64_t a_rows, const void* A,
                                 const void* B, const int32_t* offsets, const int32_t* row_index, lpgemm_type type,
                                 void* C, hipStream_t stream) {
  bool nothing;
  lpgemm_status st = check(rows, groups, N, K, a_rows, 8, LPGEMM_MAX_K_F16, 2 * K, A, B, true, offsets, row_index,
                           false, nullptr, nullptr, 1, type, C, nothing);
  if (st != LPGEMM_SUCCESS || nothing) return st;
  DeviceInfo dev;
  st = current_device(dev);
  if (st != LPGEMM_SUCCESS) return st;
  return run_grouped<KIND_F16>(args_of(rows, groups, N, a_rows, 2 * K, A, B, offsets, row_index, type, C),
                               dev.cu_count, stream);
}

lpgemm_status lpgemm_mxfp4_grouped(int64_t rows, int64_t groups, int64_t N, int64_t K, int64_t a_rows,
                                   const uint8_t* A, const uint8_t* A_scale, const uint8_t* B, const uint8_t* B_scale,
                                   const int32_t* offsets, const int32_t* row_index, lpgemm_type type, void* C,
                                   hipStream_t stream) {
  return mxfp4(rows, groups, N, K, a_rows, A, A_scale, B, B_scale, true, offsets, row_index, type, C, stream);
}

lpgemm_status lpgemm_mxfp4(int64_t M, int64_t N, int64_t K, const uint8_t* A, const uint8_t* A_scale,
                           const uint8_t* B, const uint8_t* B_scale, lpgemm_type type, void* C, hipStream_t stream) {
  return mxfp4(M, 1, N, K, M, A, A_scale, B, B_scale, false, nullptr, nullptr, type, C, stream);
}

int lpgemm_grouped_config_count(void) { return GCFG_COUNT; }

int lpgemm_force_grouped_config(int config) {
  return g_forced_grouped.exchange(config >= 0 && config < GCFG_COUNT ? config : -1);
}

int lpgemm_grouped_auto_config(int kind, int64_t rows, int64_t groups, int64_t N, int64_t K, int cu_count) {
  if ((kind != KIND_F16 && kind != KIND_I8_DEQUANT && kind != KIND_MXFP4) || cu_count < 1) return -1;
  if (rows <= 0 || groups <= 0 || N <= 0 || rows > INT32_MAX || groups > LPGEMM_MAX_GROUPS || N > INT32_MAX) return -1;
  if (K < 0 || K > INT32_MAX / 2) return -1;
  const int64_t row_bytes = kind == KIND_F16 ? 2 * K : (kind == KIND_MXFP4 ? K / 2 : K);
  return (int)choose_grouped(kind, rows, groups, N, row_bytes, cu_count);
}

}  // extern "C"
