// C entry points of the 4-bit weights with group scales
// (include/lpgemm_ffn.h).
#include "few_rows.hpp"
#include "w4_kernels.hpp"
#include "ffn.hpp"
#include "w4_tile.hpp"

using namespace lpgemm;

namespace {

bool is_16bit(lpgemm_type t) { return t == LPGEMM_F16 || t == LPGEMM_BF16; }
bool any_type(lpgemm_type t) { return is_16bit(t) || t == LPGEMM_F32; }
bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }
bool bad_group(int64_t K, int64_t group) {
  return (group != 32 && group != 64 && group != 128 && group != 256) || K % group != 0 || K > LPGEMM_MAX_K_W4;
}
// More rows, columns or tiles of a product than its kernels index.
bool too_large(int64_t M, int64_t N) {
  return M > LPGEMM_MAX_M_W4 || N > LPGEMM_MAX_N_W4 || (M + 63) / 64 * ((N + 63) / 64) >= (int64_t)1 << 24;
}
int log2_of(int64_t v) { return 63 - __builtin_clzll((unsigned long long)v); }

lpgemm_status enqueue(const void* fn, int64_t grid, void* args, hipStream_t stream) {
  void* kargs[] = {args};
  return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(256), kargs, 0, stream) == hipSuccess ? LPGEMM_SUCCESS
                                                                                             : LPGEMM_ERROR_LAUNCH;
}

// The kernels index a launch's chunks of 8 values in 32 bits; more rows than
// that go out in several launches.
int64_t rows_per_launch(int64_t chunks) { return ((int64_t)1 << 31) / chunks; }

template <typename T, bool ZEROS>
const void* quantize_kernel(int64_t group) {
  return group == 32    ? (const void*)&quantize_w4_kernel<T, 4, ZEROS>
         : group == 64  ? (const void*)&quantize_w4_kernel<T, 8, ZEROS>
         : group == 128 ? (const void*)&quantize_w4_kernel<T, 16, ZEROS>
                        : (const void*)&quantize_w4_kernel<T, 32, ZEROS>;
}

template <typename T>
const void* dequantize_kernel(lpgemm_type out) {
  return out == LPGEMM_F32   ? (const void*)&dequantize_w4_kernel<T, 0>
         : out == LPGEMM_F16 ? (const void*)&dequantize_w4_kernel<T, 1>
                             : (const void*)&dequantize_w4_kernel<T, 2>;
}

// The workspace of a plan, in bytes from its start: W4_WHOLE the weights in 16
// bits, their rows' factors and the splits' sums, W4_TILE the splits' sums.
struct W4Space {
  int64_t factors, part, total;
  W4Space(const W4Plan& plan, int64_t M, int64_t N, int64_t F, int64_t K, int cu_count) {
    const int job = F > 0 ? JOB_GATED : JOB_DOWN;
    factors = plan.way == W4_WHOLE ? (2 * N * K + 255) / 256 * 256 : 0;
    part = plan.way == W4_WHOLE && K > 0 ? factors + (4 * part_stride(job, N) + 255) / 256 * 256 : factors;
    total = part + (plan.way == W4_WHOLE ? split_bytes(plan_tiles(job, M, N, K, cu_count), job, M, N) : w4_part_bytes(plan, M, N));
  }
};

// The product through 16-bit weights.  Rounding a weight to T is what the matrix
// instructions' operands ask for: in bf16 the output is then 0.0022 from 64 bits
// (root mean square, of the output's), with exact weights 0.0017, most of which is
// the output's own rounding.  Weights in two parts, the rounded one and the rest,
// would be as good as exact ones for twice the product's time (67 of 78 us at 2048
// x 4096 x 4096).
template <typename T>
lpgemm_status run_whole(int64_t group, const W4TileArgs& w, uint8_t* ws, const W4Space& space, int64_t ws_bytes,
                        int cu_count, hipStream_t stream) {
  const int job = w.F > 0 ? JOB_GATED : JOB_DOWN;
  float *const factors = reinterpret_cast<float*>(ws + space.factors), *const part = reinterpret_cast<float*>(ws + space.part);
  TileArgs p{};
  p.A = w.X;
  p.B = ws;
  p.a_stride = w.x_stride;
  p.b_stride = 2 * (int64_t)w.K;
  p.C = p.H = w.C;
  p.out_type = w.out_type;
  p.activation = w.activation;
  p.M = w.M;
  p.N = w.N;
  p.F = w.F;
  p.K = w.K;
  if (w.K == 0) return run_tile<T>(job, p, part, ws_bytes - space.part, cu_count, stream);   // an empty sum
  p.factors = factors;
  RowsW4Args r{};
  r.codes = w.W;
  r.scales = w.scales;
  r.zeros = w.zeros;
  r.Y = ws;
  r.factors = factors;
  r.F = w.F > 0 ? w.F : w.N;
  r.rows_padded = (int)part_stride(job, w.N);
  r.rows_up = w.F > 0 ? r.rows_padded / 2 : r.rows_padded;
  r.chunks = w.K / 8;
  r.groups = w.groups;
  r.lanes_log2 = log2_of(group / 8);
  void* kargs[] = {&r};
  if (hipLaunchKernel((const void*)&rows_w4_kernel<T>, dim3((unsigned)tiles(r.rows_padded, 4), (unsigned)tiles(r.chunks, 512)),
                      dim3(256), kargs, 0, stream) != hipSuccess)
    return LPGEMM_ERROR_LAUNCH;
  return run_tile<T, true>(job, p, part, ws_bytes - space.part, cu_count, stream);
}

// The product, and (F > 0) the gated product.
lpgemm_status product(int64_t M, int64_t N, int64_t F, int64_t K, int64_t group, lpgemm_type type, int activation,
                      const void* X, int64_t x_stride, const uint8_t* codes, const void* scales, const void* zeros,
                      lpgemm_type out_type, void* C, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (bad_group(K, group) || x_stride < K || x_stride % 8 != 0 || x_stride > LPGEMM_MAX_STRIDE)
    return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  if (too_large(M, N)) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  if (M == 0 || N == 0) return LPGEMM_SUCCESS;
  if (!C || (K > 0 && (!X || !codes || !scales))) return LPGEMM_ERROR_INVALID_VALUE;
  if (!aligned16(C) || (K > 0 && (!aligned16(X) || !aligned16(codes) || !aligned2(scales) || !aligned2(zeros))))
    return LPGEMM_ERROR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return LPGEMM_ERROR_MISALIGNED;
  DeviceInfo dev;
  const lpgemm_status st = current_device(dev);
  if (st != LPGEMM_SUCCESS) return st;
  const W4Plan plan = plan_w4(M, N, K, dev.cu_count);
  const W4Space space(plan, M, N, F, K, dev.cu_count);
  const int64_t need = space.total;
  if (need > 0 && (!workspace || workspace_bytes < need)) return LPGEMM_ERROR_INVALID_VALUE;
  const int w4 = group == 32 ? 1 : group == 64 ? 2 : 4;
  if (plan.way == W4_FEW_ROWS) {
    FewRowsArgs p{};
    p.X = static_cast<const uint8_t*>(X);
    p.W = codes;
    p.scales = static_cast<const uint16_t*>(scales);
    p.zeros = static_cast<const uint16_t*>(zeros);
    p.C = static_cast<uint8_t*>(C);
    p.out_type = out_type;
    p.M = (int)M;
    p.N = (int)N;
    p.F = (int)F;
    p.K = (int)K;
    p.activation = activation;
    p.x_stride = (int)(2 * x_stride);
    p.row_bytes = (int)(K / 2);
    p.groups = (int)(K / group);
    p.group_shift = group == 256 ? 1 : 0;
    return type == LPGEMM_F16 ? run_few_rows<TypeF16>(p, w4, dev.cu_count, stream)
                              : run_few_rows<TypeBF16>(p, w4, dev.cu_count, stream);
  }
  W4TileArgs p{};
  p.X = static_cast<const uint8_t*>(X);
  p.W = codes;
  p.scales = static_cast<const uint16_t*>(scales);
  p.zeros = static_cast<const uint16_t*>(zeros);
  p.C = static_cast<uint8_t*>(C);
  p.out_type = out_type;
  p.M = (int)M;
  p.N = (int)N;
  p.F = (int)F;
  p.K = (int)K;
  p.activation = activation;
  p.x_stride = (int)(2 * x_stride);
  p.row_bytes = (int)(K / 2);
  p.groups = (int)(K / group);
  p.group_shift = log2_of(group);
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  p.part = reinterpret_cast<float*>(ws + space.part);
  if (plan.way == W4_WHOLE)
    return type == LPGEMM_F16 ? run_whole<TypeF16>(group, p, ws, space, workspace_bytes, dev.cu_count, stream)
                              : run_whole<TypeBF16>(group, p, ws, space, workspace_bytes, dev.cu_count, stream);
  if (type == LPGEMM_F16)
    return w4 == 1   ? run_w4_tile<TypeF16, 1>(plan, p, stream)
           : w4 == 2 ? run_w4_tile<TypeF16, 2>(plan, p, stream)
                     : run_w4_tile<TypeF16, 4>(plan, p, stream);
  return w4 == 1   ? run_w4_tile<TypeBF16, 1>(plan, p, stream)
         : w4 == 2 ? run_w4_tile<TypeBF16, 2>(plan, p, stream)
                   : run_w4_tile<TypeBF16, 4>(plan, p, stream);
}

}  // namespace

extern "C" {

lpgemm_status lpgemm_quantize_w4(int64_t N, int64_t K, int64_t group, lpgemm_type type, const void* W,
                                 int64_t w_stride, uint8_t* codes, void* scales, void* zeros, hipStream_t stream) {
  if (N < 0 || K < 0 || group < 0 || N > INT32_MAX || !is_16bit(type)) return LPGEMM_ERROR_INVALID_VALUE;
  if (bad_group(K, group) || w_stride < K || w_stride % 8 != 0) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  if (N == 0 || K == 0) return LPGEMM_SUCCESS;
  if (!W || !codes || !scales) return LPGEMM_ERROR_INVALID_VALUE;
  if (!aligned16(W) || !aligned16(codes) || !aligned2(scales) || !aligned2(zeros)) return LPGEMM_ERROR_MISALIGNED;
  DeviceInfo dev;
  lpgemm_status st = current_device(dev);
  if (st != LPGEMM_SUCCESS) return st;
  const void* fn = type == LPGEMM_F16
                       ? (zeros ? quantize_kernel<TypeF16, true>(group) : quantize_kernel<TypeF16, false>(group))
                       : (zeros ? quantize_kernel<TypeBF16, true>(group) : quantize_kernel<TypeBF16, false>(group));
  const int64_t chunks = K / 8, groups = K / group, most = rows_per_launch(chunks);
  for (int64_t r = 0; r < N && st == LPGEMM_SUCCESS; r += most) {
    const int64_t n = N - r < most ? N - r : most;
    QuantW4Args p{};
    p.W = static_cast<const uint8_t*>(W) + 2 * r * w_stride;
    p.codes = codes + r * (K / 2);
    p.scales = static_cast<uint16_t*>(scales) + r * groups;
    p.zeros = zeros ? static_cast<uint16_t*>(zeros) + r * groups : nullptr;
    p.w_stride = 2 * w_stride;
    p.chunks = (uint32_t)chunks;
    p.total = (uint32_t)(n * chunks);
    st = enqueue(fn, (n * chunks + 255) / 256, &p, stream);
  }
  return st;
}

lpgemm_status lpgemm_dequantize_w4(int64_t N, int64_t K, int64_t group, lpgemm_type type, const uint8_t* codes,
                                   const void* scales, const void* zeros, lpgemm_type out_type, void* Y,
                                   hipStream_t stream) {
  if (N < 0 || K < 0 || group < 0 || N > INT32_MAX || !is_16bit(type) || !any_type(out_type))
    return LPGEMM_ERROR_INVALID_VALUE;
  if (bad_group(K, group)) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  if (N == 0 || K == 0) return LPGEMM_SUCCESS;
  if (!codes || !scales || !Y) return LPGEMM_ERROR_INVALID_VALUE;
  if (!aligned16(codes) || !aligned2(scales) || !aligned2(zeros) || !aligned16(Y)) return LPGEMM_ERROR_MISALIGNED;
  DeviceInfo dev;
  lpgemm_status st = current_device(dev);
  if (st != LPGEMM_SUCCESS) return st;
  const void* fn = type == LPGEMM_F16 ? dequantize_kernel<TypeF16>(out_type) : dequantize_kernel<TypeBF16>(out_type);
  const int64_t chunks = K / 8, groups = K / group, most = rows_per_launch(chunks);
  const int64_t size = out_type == LPGEMM_F32 ? 4 : 2;
  for (int64_t r = 0; r < N && st == LPGEMM_SUCCESS; r += most) {
    const int64_t n = N - r < most ? N - r : most;
    DequantW4Args p{};
    p.codes = codes + r * (K / 2);
    p.scales = static_cast<const uint16_t*>(scales) + r * groups;
    p.zeros = zeros ? static_cast<const uint16_t*>(zeros) + r * groups : nullptr;
    p.Y = static_cast<uint8_t*>(Y) + r * K * size;
    p.total = (uint32_t)(n * chunks);
    p.lanes_log2 = log2_of(group / 8);
    st = enqueue(fn, (n * chunks + 255) / 256, &p, stream);
  }
  return st;
}

int64_t lpgemm_w4_workspace(int64_t M, int64_t N, int64_t K, int64_t group, int gated) {
  if (M < 0 || N < 0 || K < 0 || too_large(M, N) || bad_group(K, group) || (gated && N % 2 != 0)) return -1;
  if (M == 0 || N == 0) return 0;
  DeviceInfo dev;
  if (current_device(dev) != LPGEMM_SUCCESS) return -1;
  const W4Plan plan = plan_w4(M, N, K, dev.cu_count);
  return W4Space(plan, M, N, gated ? N / 2 : 0, K, dev.cu_count).total;
}

lpgemm_status lpgemm_w4(int64_t M, int64_t N, int64_t K, int64_t group, lpgemm_type type, const void* X,
                        int64_t x_stride, const uint8_t* codes, const void* scales, const void* zeros,
                        lpgemm_type out_type, void* C, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  if (M < 0 || N < 0 || K < 0 || group < 0 || M > INT32_MAX || N > INT32_MAX || !is_16bit(type) ||
      !any_type(out_type) || workspace_bytes < 0)
    return LPGEMM_ERROR_INVALID_VALUE;
  return product(M, N, 0, K, group, type, 0, X, x_stride, codes, scales, zeros, out_type, C, workspace,
                 workspace_bytes, stream);
}

lpgemm_status lpgemm_gated_w4(int64_t M, int64_t F, int64_t K, int64_t group, lpgemm_type type,
                              lpgemm_activation activation, const void* X, int64_t x_stride, const uint8_t* codes,
                              const void* scales, const void* zeros, lpgemm_type out_type, void* H, void* workspace,
                              int64_t workspace_bytes, hipStream_t stream) {
  if (M < 0 || F < 0 || K < 0 || group < 0 || M > INT32_MAX || F > INT32_MAX || !is_16bit(type) ||
      !any_type(out_type) || (activation != LPGEMM_SILU && activation != LPGEMM_GELU) || workspace_bytes < 0)
    return LPGEMM_ERROR_INVALID_VALUE;
  return product(M, 2 * F, F, K, group, type, activation, X, x_stride, codes, scales, zeros, out_type, H, workspace,
                 workspace_bytes, stream);
}

}  // extern "C"
