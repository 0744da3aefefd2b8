// Layout probes of the 16-bit kernels' instructions: single-instruction
// kernels that pin, on the device, the lane layouts that half_types.hpp
// states.  Test infrastructure only (tests/test_gpu_half_layouts.py).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../precision_dense_gemm_02_amd/csrc/half_types.hpp"
#include "../../precision_dense_gemm_02_amd/csrc/w4_tile_kernels.hpp"

using namespace lpgemm;

namespace {

// A: 32 x 16, Bt: 32 x 16 values of T; C = A . B, 32 x 32 binary32
template <typename T>
__global__ __launch_bounds__(64) void k_mfma32(const uint16_t* A, const uint16_t* Bt, float* C) {
  const int l = threadIdx.x;
  const i32x4 a = *(const i32x4*)(A + (l & 31) * 16 + 8 * (l >> 5));
  const i32x4 b = *(const i32x4*)(Bt + (l & 31) * 16 + 8 * (l >> 5));
  f32x16 acc = {};
  acc = mfma32<T>(a, b, acc);
  for (int e = 0; e < 16; ++e) C[(8 * (e >> 2) + 4 * (l >> 5) + (e & 3)) * 32 + (l & 31)] = acc[e];
}

// A: 16 x 32, Bt: 16 x 32 values of T; C = A . B, 16 x 16 binary32
template <typename T>
__global__ __launch_bounds__(64) void k_mfma16(const uint16_t* A, const uint16_t* Bt, float* C) {
  const int l = threadIdx.x;
  const i32x4 a = *(const i32x4*)(A + (l & 15) * 32 + 8 * (l >> 4));
  const i32x4 b = *(const i32x4*)(Bt + (l & 15) * 32 + 8 * (l >> 4));
  f32x4 acc = {};
  acc = mfma16<T>(a, b, acc);
  for (int e = 0; e < 4; ++e) C[(4 * (l >> 4) + e) * 16 + (l & 15)] = acc[e];
}

// 1 KiB into LDS, then one transposing read per lane at the byte offset
// addr[lane]; out: 4 values per lane
__global__ __launch_bounds__(64) void k_read_transposed(const uint16_t* in, const int* addr, uint16_t* out) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[1024];
  const int l = threadIdx.x;
  *(i32x4*)(lds + 16 * l) = *(const i32x4*)(in + 8 * l);
  __syncthreads();
  const u32x2 v = lds_read_transposed16(lds_address(lds) + addr[l]);
  *(u32x2*)(out + 4 * l) = v;
}

// four words per lane, out: the same after transpose_rows
__global__ __launch_bounds__(64) void k_transpose_rows(const uint32_t* in, const int*, uint32_t* out) {
  const int l = threadIdx.x;
  *(u32x4*)(out + 4 * l) = transpose_rows(*(const u32x4*)(in + 4 * l));
}

// 16-bit values at the byte offsets offset[lane] of 128 values, straight into
// LDS; out: the 64 words there, which held ones
__global__ __launch_bounds__(64) void k_dma2(const uint16_t* in, const int* offset, uint32_t* out) {
  __shared__ __attribute__((aligned(16))) uint32_t lds[64];
  const int l = threadIdx.x;
  lds[l] = 0xffffffffu;
  __syncthreads();
  lds_dma_2(make_rsrc(in, 256), lds_address((uint8_t*)lds), (uint32_t)offset[l]);
  wait_vmcnt<0>();
  __syncthreads();
  out[l] = lds[l];
}

int launch1(const void* fn, void** args, hipStream_t s) {
  return hipLaunchKernel(fn, dim3(1), dim3(64), args, 0, s) == hipSuccess ? 0 : 1;
}

}  // namespace

extern "C" {

int probe_mfma32(int bf16, const uint16_t* A, const uint16_t* Bt, float* C, hipStream_t s) {
  void* a[] = {&A, &Bt, &C};
  return launch1(bf16 ? (const void*)&k_mfma32<TypeBF16> : (const void*)&k_mfma32<TypeF16>, a, s);
}

int probe_mfma16(int bf16, const uint16_t* A, const uint16_t* Bt, float* C, hipStream_t s) {
  void* a[] = {&A, &Bt, &C};
  return launch1(bf16 ? (const void*)&k_mfma16<TypeBF16> : (const void*)&k_mfma16<TypeF16>, a, s);
}

int probe_read_transposed(int, const uint16_t* in, const int* addr, uint16_t* out, hipStream_t s) {
  void* a[] = {&in, &addr, &out};
  return launch1((const void*)&k_read_transposed, a, s);
}

int probe_transpose_rows(int, const uint32_t* in, const int* unused, uint32_t* out, hipStream_t s) {
  void* a[] = {&in, &unused, &out};
  return launch1((const void*)&k_transpose_rows, a, s);
}

int probe_dma2(int, const uint16_t* in, const int* offset, uint32_t* out, hipStream_t s) {
  void* a[] = {&in, &offset, &out};
  return launch1((const void*)&k_dma2, a, s);
}

}  // extern "C"
