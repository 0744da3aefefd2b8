// The two 16-bit operand types of the feed-forward and 4-bit-weight kernels:
// their matrix instructions, their widening and rounding, and the two lane
// exchanges that bring operands into the matrix instructions' layout.
#pragma once

#include "gemm_kernels.hpp"
#include "row_kernels.hpp"

namespace lpgemm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <typename T>
constexpr bool kIsF16 = std::is_same<T, TypeF16>::value;

// 32 x 32 x 16: lane l holds row (column) l % 32, k = 8 (l / 32) .. + 7;
// element e of the sum is row 8 (e / 4) + 4 (l / 32) + e % 4, column l % 32.
template <typename T>
__device__ __forceinline__ f32x16 mfma32(const i32x4& a, const i32x4& b, const f32x16& c) {
  if constexpr (kIsF16<T>)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// 16 x 16 x 32: lane l holds row (column) l % 16, k = 8 (l / 16) .. + 7;
// element e of the sum is row 4 (l / 16) + e, column l % 16.
template <typename T>
__device__ __forceinline__ f32x4 mfma16(const i32x4& a, const i32x4& b, const f32x4& c) {
  if constexpr (kIsF16<T>)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Transposing LDS read of 16-bit values: within each group of 16 lanes, lane c
// receives value c of the four 16-value rows that lanes 4 b .. 4 b + 3 address
// (8 bytes each), in order of b.
__device__ __forceinline__ u32x2 lds_read_transposed16(uint32_t lds_addr) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)lds_addr));
}

// Four words of four 16-lane rows, transposed: word j of row q becomes what
// word q of row j was.
__device__ __forceinline__ u32x4 transpose_rows(const u32x4& d) {
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(d.x, d.z, false, false));
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(d.y, d.w, false, false));
  const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a.x, b.x, false, false));
  const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a.y, b.y, false, false));
  return u32x4{lo.x, lo.y, hi.x, hi.y};
}

template <typename T>
__device__ __forceinline__ float widen1(uint16_t bits) {
  if constexpr (kIsF16<T>) return (float)__builtin_bit_cast(_Float16, bits);
  else return __builtin_bit_cast(float, (uint32_t)bits << 16);
}

// Eight binary32 values rounded once, to nearest even.
template <typename T>
__device__ __forceinline__ i32x4 narrow8(const float (&v)[8]) {
  const f32x8 w = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
  return __builtin_bit_cast(i32x4, __builtin_convertvector(w, typename T::x8));
}
template <typename T>
__device__ __forceinline__ uint16_t narrow1(float v) {
  if constexpr (kIsF16<T>) return __builtin_bit_cast(uint16_t, (_Float16)v);
  else return __builtin_bit_cast(uint16_t, (__bf16)v);
}

}  // namespace lpgemm
