// C entry points of the row kernels (include/lpgemm_moe.h): residual +
// RMSNorm and silu(gate) * up with int8 rows, MXFP4 quantisation and its
// inverse.
#include "../../include/lpgemm_moe.h"
#include "dispatch.hpp"
#include "row_kernels.hpp"

using namespace lpgemm;

namespace {

bool is_16bit(lpgemm_type t) { return t == LPGEMM_F16 || t == LPGEMM_BF16; }

lpgemm_status enqueue(const void* fn, int64_t grid, int threads, void* args, hipStream_t stream) {
  void* kargs[] = {args};
  return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(threads), kargs, 0, stream) == hipSuccess
             ? LPGEMM_SUCCESS
             : LPGEMM_ERROR_LAUNCH;
}

// The kernel for rows of K values: in registers up to 32768 values, with the
// wavefronts per row that leave a lane one to four chunks.  More of them lose
// to the join and to idle lanes, fewer to the latency of a lane's loads
// (bfloat16, us on one MI355X with 1, 2, 4, 8 and 16 wavefronts; norm, 8192
// rows of 512: 9.7 10.8 14.8 23.5 45.3; of 1024: 15.1 15.6 18.5 27.0 49.8; of
// 4096: 50.2 46.8 44.5 46.1 60.4; of 8192: - 89.2 86.0 84.6 90.3; of 14336: -
// - 148 146 146; activation, 8192 rows of 14336: - - 112 113 106; 16 rows: - -
// 5.1 4.4 4.4; 8192 rows of 32768: - - - 245 236, and 337 in two passes).
template <typename T, bool NORM>
lpgemm_status launch_rows(RowArgs& p, hipStream_t stream) {
  const int K = p.K;
  const void* fn;
  int waves, rows = 1;   // wavefronts of a workgroup, its rows
  if (K == 0 || K > 32768) fn = (const void*)&rows_int8_long<T, NORM>, waves = 16;
  else if (K <= 512) fn = (const void*)&rows_int8_regs<T, NORM, 1, 1>, waves = rows = 4;
  else if (K <= 1024) fn = (const void*)&rows_int8_regs<T, NORM, 2, 1>, waves = 2;
  else if (K <= 2048) fn = (const void*)&rows_int8_regs<T, NORM, 4, 1>, waves = 4;
  else if (K <= 4096) fn = (const void*)&rows_int8_regs<T, NORM, 4, 2>, waves = 4;
  else if (K <= 8192) fn = (const void*)&rows_int8_regs<T, NORM, 8, 2>, waves = 8;
  else if (K <= 16384 && NORM) fn = (const void*)&rows_int8_regs<T, NORM, 8, 4>, waves = 8;
  else if (K <= 16384) fn = (const void*)&rows_int8_regs<T, NORM, 16, 2>, waves = 16;
  else fn = (const void*)&rows_int8_regs<T, NORM, 16, 4>, waves = 16;
  return enqueue(fn, ((int64_t)p.M + rows - 1) / rows, 64 * waves, &p, stream);
}

// A grid holds less than 2^32 threads: more rows than this go out in several
// launches.
constexpr int64_t kRowsPerLaunch = (int64_t)1 << 21;

template <typename T, bool NORM>
lpgemm_status run_rows(RowArgs p, int64_t M, hipStream_t stream) {
  lpgemm_status st = LPGEMM_SUCCESS;
  for (int64_t r = 0; r < M && st == LPGEMM_SUCCESS; r += kRowsPerLaunch) {
    p.M = (int)(M - r < kRowsPerLaunch ? M - r : kRowsPerLaunch);
    st = launch_rows<T, NORM>(p, stream);
    p.X += kRowsPerLaunch * p.x_stride;
    if (p.R) p.R += kRowsPerLaunch * p.r_stride;
    if (p.H) p.H += kRowsPerLaunch * p.h_stride;
    p.Q += kRowsPerLaunch * p.K;
    p.scale += kRowsPerLaunch;
  }
  return st;
}

bool bad_stride(int64_t stride, int64_t least) { return stride < least || stride % 8 != 0; }

}  // namespace

extern "C" {

lpgemm_status lpgemm_add_rmsnorm_quantize(int64_t M, int64_t K, lpgemm_type type, const void* X, int64_t x_stride,
                                          const void* R, int64_t r_stride, const void* weight, float eps, void* H,
                                          int64_t h_stride, int8_t* Q, float* row_scale, hipStream_t stream) {
  if (M < 0 || K < 0 || M > INT32_MAX || !is_16bit(type) || !(eps >= 0.f)) return LPGEMM_ERROR_INVALID_VALUE;
  if (K % 8 != 0 || K > LPGEMM_MAX_K_QUANT) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  if (bad_stride(x_stride, K) || (R && bad_stride(r_stride, K)) || (H && bad_stride(h_stride, K)))
    return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  if (M == 0) return LPGEMM_SUCCESS;
  if (!row_scale || (K > 0 && (!X || !weight || !Q))) return LPGEMM_ERROR_INVALID_VALUE;
  if (!aligned4(row_scale)) return LPGEMM_ERROR_MISALIGNED;
  if (K > 0 && (!aligned16(X) || !aligned16(R) || !aligned16(weight) || !aligned16(H) || !aligned16(Q)))
    return LPGEMM_ERROR_MISALIGNED;
  DeviceInfo dev;   // (fails on another GPU than this library is built for)
  const lpgemm_status st = current_device(dev);
  if (st != LPGEMM_SUCCESS) return st;
  RowArgs p{};
  p.X = static_cast<const uint8_t*>(X);
  p.R = static_cast<const uint8_t*>(R);
  p.weight = static_cast<const uint8_t*>(weight);
  p.H = static_cast<uint8_t*>(H);
  p.Q = Q;
  p.scale = row_scale;
  p.x_stride = 2 * x_stride;
  p.r_stride = 2 * r_stride;
  p.h_stride = 2 * h_stride;
  p.K = (int)K;
  p.eps = eps;
  return type == LPGEMM_F16 ? run_rows<TypeF16, true>(p, M, stream)
                            : run_rows<TypeBF16, true>(p, M, stream);
}

lpgemm_status lpgemm_silu_mul_quantize(int64_t M, int64_t K, lpgemm_type type, const void* X, int64_t x_stride,
                                       int8_t* Q, float* row_scale, hipStream_t stream) {
  if (M < 0 || K < 0 || M > INT32_MAX || !is_16bit(type)) return LPGEMM_ERROR_INVALID_VALUE;
  if (K % 8 != 0 || K > LPGEMM_MAX_K_QUANT) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  if (bad_stride(x_stride, 2 * K)) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  if (M == 0) return LPGEMM_SUCCESS;
  if (!row_scale || (K > 0 && (!X || !Q))) return LPGEMM_ERROR_INVALID_VALUE;
  if (!aligned4(row_scale)) return LPGEMM_ERROR_MISALIGNED;
  if (K > 0 && (!aligned16(X) || !aligned16(Q))) return LPGEMM_ERROR_MISALIGNED;
  DeviceInfo dev;   // (fails on another GPU than this library is built for)
  const lpgemm_status st = current_device(dev);
  if (st != LPGEMM_SUCCESS) return st;
  RowArgs p{};
  p.X = static_cast<const uint8_t*>(X);
  p.Q = Q;
  p.scale = row_scale;
  p.x_stride = 2 * x_stride;
  p.K = (int)K;
  return type == LPGEMM_F16 ? run_rows<TypeF16, false>(p, M, stream)
                            : run_rows<TypeBF16, false>(p, M, stream);
}

// The MXFP4 kernels index a launch's chunks of 8 values in 32 bits; more
// rows than that go out in several launches.
static int64_t rows_per_launch(int64_t chunks) { return ((int64_t)1 << 31) / chunks; }

// Two chunks of 8 values per lane, for twice the loads in flight, from 2^25
// values on (from bfloat16 and back, us with one chunk and with two: 14336
// x 4096 31.3 and 29.8, inverse 40.0 and 30.3; with a kernel that writes the
// values before or reads them after, 59.5 and 57.5, 68.3 and 59.5; 4096 x 4096
// 20.9 and 21.5, 20.8 and 23.4).
static bool two_chunks(int64_t rows, int64_t chunks) { return rows * chunks >= (int64_t)1 << 22; }
static int64_t tiles_of(int64_t n, int64_t t) { return (n + t - 1) / t; }

lpgemm_status lpgemm_quantize_mxfp4(int64_t rows, int64_t K, lpgemm_type type, const void* X, int64_t x_stride,
                                    uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  if (rows < 0 || K < 0 || rows > INT32_MAX || !is_16bit(type)) return LPGEMM_ERROR_INVALID_VALUE;
  if (K % 32 != 0 || K > LPGEMM_MAX_K_MXFP4 || bad_stride(x_stride, K)) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  if (rows == 0 || K == 0) return LPGEMM_SUCCESS;
  if (!X || !codes || !scales) return LPGEMM_ERROR_INVALID_VALUE;
  if (!aligned16(X) || !aligned16(codes) || !aligned16(scales)) return LPGEMM_ERROR_MISALIGNED;
  DeviceInfo dev;
  lpgemm_status st = current_device(dev);
  if (st != LPGEMM_SUCCESS) return st;
  const int64_t chunks = K / 8, stride = LPGEMM_MXFP4_SCALE_STRIDE(K), most = rows_per_launch(chunks);
  const bool two = two_chunks(rows, chunks);
  const void* fn = type == LPGEMM_F16
                       ? (two ? (const void*)&quantize_mxfp4_kernel<TypeF16, 2> : (const void*)&quantize_mxfp4_kernel<TypeF16, 1>)
                       : (two ? (const void*)&quantize_mxfp4_kernel<TypeBF16, 2> : (const void*)&quantize_mxfp4_kernel<TypeBF16, 1>);
  for (int64_t r = 0; r < rows && st == LPGEMM_SUCCESS; r += most) {
    const int64_t n = rows - r < most ? rows - r : most;
    Mxfp4Args p{};
    p.X = static_cast<const uint8_t*>(X) + 2 * r * x_stride;
    p.codes = codes + r * (K / 2);
    p.scales = scales + r * stride;
    p.x_stride = 2 * x_stride;
    p.chunks = (int)chunks;
    p.scale_stride = (int)stride;
    p.total = (uint32_t)(n * chunks);
    st = enqueue(fn, tiles_of(n * chunks, two ? 512 : 256), 256, &p, stream);
  }
  return st;
}

lpgemm_status lpgemm_dequantize_mxfp4(int64_t rows, int64_t K, const uint8_t* codes, const uint8_t* scales,
                                      lpgemm_type type, void* Y, hipStream_t stream) {
  if (rows < 0 || K < 0 || rows > INT32_MAX || !(is_16bit(type) || type == LPGEMM_F32))
    return LPGEMM_ERROR_INVALID_VALUE;
  if (K % 32 != 0 || K > LPGEMM_MAX_K_MXFP4) return LPGEMM_ERROR_UNSUPPORTED_SHAPE;
  if (rows == 0 || K == 0) return LPGEMM_SUCCESS;
  if (!codes || !scales || !Y) return LPGEMM_ERROR_INVALID_VALUE;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(Y)) return LPGEMM_ERROR_MISALIGNED;
  DeviceInfo dev;
  lpgemm_status st = current_device(dev);
  if (st != LPGEMM_SUCCESS) return st;
  const int64_t chunks = K / 8, stride = LPGEMM_MXFP4_SCALE_STRIDE(K), most = rows_per_launch(chunks);
  const bool two = two_chunks(rows, chunks);
  const void* fn =
      type == LPGEMM_F32   ? (two ? (const void*)&dequantize_mxfp4_kernel<0, 2> : (const void*)&dequantize_mxfp4_kernel<0, 1>)
      : type == LPGEMM_F16 ? (two ? (const void*)&dequantize_mxfp4_kernel<1, 2> : (const void*)&dequantize_mxfp4_kernel<1, 1>)
                           : (two ? (const void*)&dequantize_mxfp4_kernel<2, 2> : (const void*)&dequantize_mxfp4_kernel<2, 1>);
  const int64_t size = type == LPGEMM_F32 ? 4 : 2;
  for (int64_t r = 0; r < rows && st == LPGEMM_SUCCESS; r += most) {
    const int64_t n = rows - r < most ? rows - r : most;
    Dequant4Args p{};
    p.codes = codes + r * (K / 2);
    p.scales = scales + r * stride;
    p.Y = static_cast<uint8_t*>(Y) + r * K * size;
    p.chunks = (int)chunks;
    p.scale_stride = (int)stride;
    p.total = (uint32_t)(n * chunks);
    st = enqueue(fn, tiles_of(n * chunks, two ? 512 : 256), 256, &p, stream);
  }
  return st;
}

}  // extern "C"
