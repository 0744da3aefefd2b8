// 4-bit weights with group scales: quantisation, its inverse, and the inverse
// that a product of 16-bit weights reads.
#pragma once

#include "half_types.hpp"

namespace lpgemm {

struct QuantW4Args {
  const uint8_t* W;
  uint8_t* codes;
  uint16_t* scales;
  uint16_t* zeros;     // null: none
  int64_t w_stride;    // bytes
  uint32_t chunks;     // chunks of 8 values per row
  uint32_t total;      // ... in all rows
};

// A lane holds 8 values; LANES lanes a group.  The quotients are those of the
// division, from one reciprocal per group: with r = RN(1 / s) and q = RN(w r),
// RN(q + r (w - q s)) is the correctly rounded quotient (Markstein), three
// operations instead of ten.
//
// 14336 x 4096 bf16, groups of 128: 37 to 42 us, 3.6 to 4.0 TB/s (41 with zeros);
// the inverse to fp32 41 to 52 us, 5.2 to 6.5 TB/s (part of its output stays in the
// caches).  The quantisation spends its time on the 25 vector operations that it
// has for each value, not on memory.  That is not the least: a branch per code, a
// zero that is added where there is none, masks and shifts apart and a division
// per lane are in them.
template <typename T, int LANES, bool ZEROS>
__global__ __launch_bounds__(256) void quantize_w4_kernel(QuantW4Args p) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= p.total) return;   // (whole groups: rows are whole groups)
  const uint32_t row = i / p.chunks, chunk = i - row * p.chunks;
  const i32x4 raw = *(const i32x4*)(p.W + row * p.w_stride + 16 * (int64_t)chunk);
  const f32x8 w = widen<T>(raw);
  uint32_t top = 0;            // largest magnitude, as bits: a NaN is larger than everything
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float v = w[e];   // (a bit cast of a vector's element would take the first)
    top = max(top, __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu);
    if constexpr (ZEROS) {
      lo = fminf(lo, v);
      hi = fmaxf(hi, v);
    }
  }
#pragma unroll
  for (int off = 1; off < LANES; off <<= 1) {
    top = max(top, (uint32_t)__shfl_xor((int)top, off));
    if constexpr (ZEROS) {
      lo = fminf(lo, __shfl_xor(lo, off));
      hi = fmaxf(hi, __shfl_xor(hi, off));
    }
  }
  const bool finite = top < kInfBits;
  const float span = ZEROS ? hi - lo : __builtin_bit_cast(float, top);
  uint16_t sbits = finite ? narrow1<T>(span >= kTinyRow ? span / (ZEROS ? 15.f : 7.f) : 0.f) : narrow1<T>(__builtin_nanf(""));
  const float s = widen1<T>(sbits);
  const bool live = finite && s > 0.f && s < __builtin_inff();
  const float r = live ? 1.f / s : 0.f;
  auto steps = [&](float v) {
    const float q = __fmul_rn(v, r);
    return __builtin_rintf(__builtin_fmaf(__builtin_fmaf(-q, s, v), r, q));
  };
  const float zero = ZEROS && live ? fminf(fmaxf(-8.f - steps(lo), -8.f), 7.f) : 0.f;
  uint32_t packed = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float code = live ? fminf(fmaxf(steps(w[e]) + zero, -8.f), 7.f) : 0.f;
    packed |= ((uint32_t)(int)code & 15u) << (4 * e);
  }
  *(uint32_t*)(p.codes + 4 * (int64_t)i) = packed;
  if (threadIdx.x % LANES == 0) {
    const uint32_t group = i / LANES;
    p.scales[group] = sbits;
    if constexpr (ZEROS) p.zeros[group] = narrow1<T>(zero);
  }
}

struct DequantW4Args {
  const uint8_t* codes;
  const uint16_t* scales;
  const uint16_t* zeros;   // null: none
  uint8_t* Y;
  uint32_t total;          // chunks of 8 values
  int lanes_log2;          // chunks per group
};

// A lane turns 8 codes (4 bytes) into 8 values.  OUT: lpgemm_type of Y.
template <typename T, int OUT>
__global__ __launch_bounds__(256) void dequantize_w4_kernel(DequantW4Args p) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= p.total) return;
  const uint32_t packed = *(const uint32_t*)(p.codes + 4 * (int64_t)i);
  const uint32_t group = i >> p.lanes_log2;
  const float s = widen1<T>(p.scales[group]);
  const float z = p.zeros ? widen1<T>(p.zeros[group]) : 0.f;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __fmul_rn((float)((int)(packed << (28 - 4 * e)) >> 28) - z, s);
  if constexpr (OUT == 0) {
    f32x4* y = (f32x4*)(p.Y + 32 * (int64_t)i);
    y[0] = f32x4{v[0], v[1], v[2], v[3]};
    y[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else if constexpr (OUT == 1) {
    *(i32x4*)(p.Y + 16 * (int64_t)i) = narrow8<TypeF16>(v);
  } else {
    *(i32x4*)(p.Y + 16 * (int64_t)i) = narrow8<TypeBF16>(v);
  }
}

struct RowsW4Args {
  const uint8_t* codes;
  const uint16_t* scales;
  const uint16_t* zeros;   // null: none
  uint8_t* Y;
  float* factors;          // one per row, the up projection's from rows_up on
  int F;                   // gated: rows of each projection, else N
  int rows_up;             // F rounded up to 8
  int rows_padded;         // ... of both projections
  int chunks;              // of 8 values per row
  int groups;              // per row
  int lanes_log2;          // chunks per group
};

// Weights as values of T, each rounded once, for a product behind them.  A
// weight may lie past T's range (a scale of 5000, code 7 and a zero of -7, in
// binary16), where rounding would make it an infinity and the sums with it:
// such a row is divided by a power of two, factors[row], which its sums are
// multiplied by again.  |weight| < 2^(a + b) for |scale| < 2^a and |zero| + 8 <
// 2^b, the largest a + b of a row's groups decides; most rows have factor 1 and
// the values that dequantize_w4_kernel gives.  Infinite and NaN scales and zeros
// stay out of the choice and go into their group's values.
//
// A wave takes 4096 values of a row and finds the row's factor itself, behind
// the loads of its codes and their scales: 4096 x 4096 in groups of 128 8.7 us, 14336
// x 4096 in groups of 64 with zeros 25.1 (dequantize_w4_kernel, without factors, 8.4
// and 23.2).  With the factors' way into the sums a product of 2048 x 4096 x 4096
// takes 79 us instead of 78, the smallest ones 0.8 us more.
template <typename T>
__global__ __launch_bounds__(256) void rows_w4_kernel(RowsW4Args p) {
  constexpr int kMost = kIsF16<T> ? 15 : 127;   // |weight| below 2^kMost is in range after rounding
  const int lane = threadIdx.x & 63;
  const int at = blockIdx.x * 4 + (threadIdx.x >> 6);   // place among the factors
  const bool up = at >= p.rows_up;
  const int in_half = up ? at - p.rows_up : at;
  if (at >= p.rows_padded) return;
  if (in_half >= p.F) {                                  // (between the projections and behind them)
    if (blockIdx.y == 0 && lane == 0) p.factors[at] = 1.f;
    return;
  }
  const int64_t row = up ? p.F + in_half : in_half;
  constexpr int kEach = 8;
  const int first = blockIdx.y * (64 * kEach) + lane;
  const uint32_t* const codes = (const uint32_t*)p.codes + row * p.chunks;
  const uint16_t* const scales = p.scales + row * p.groups;
  const uint16_t* const zeros = p.zeros ? p.zeros + row * p.groups : nullptr;
  auto exponent = [](float v) { return (int)(__builtin_bit_cast(uint32_t, v) >> 23 & 255) - 126; };   // |v| < 2^it
  auto power = [](int n) { return __builtin_bit_cast(float, (uint32_t)(127 + n) << 23); };
  auto run = [&](auto whole_c) __attribute__((always_inline)) {   // all of the wave's places hold chunks
    constexpr bool whole = decltype(whole_c)::value;
    uint32_t packed[kEach];
    uint16_t scale[kEach], zero[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int c = first + 64 * i;
      if (!whole && c >= p.chunks) break;
      packed[i] = codes[c];
      scale[i] = scales[c >> p.lanes_log2];
      zero[i] = zeros ? zeros[c >> p.lanes_log2] : 0;
    }
    int most = -1000;
    for (int g = lane; g < p.groups; g += 64) {
      const int a = exponent(widen1<T>(scales[g])), b = exponent(zeros ? __builtin_fabsf(widen1<T>(zeros[g])) + 8.f : 8.f);
      if (a < 129 && b < 129) most = max(most, a + b);     // (129: infinities and NaN)
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) most = max(most, __shfl_xor(most, off));
    const int e = min(max(most - kMost, 0), 126);
    if (blockIdx.y == 0 && lane == 0) p.factors[at] = power(e);
    const float down = power(-e);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int c = first + 64 * i;
      if (!whole && c >= p.chunks) break;
      const float s = __fmul_rn(widen1<T>(scale[i]), down), z = widen1<T>(zero[i]);
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __fmul_rn((float)((int)(packed[i] << (28 - 4 * k)) >> 28) - z, s);
      *(i32x4*)(p.Y + 16 * (row * p.chunks + c)) = narrow8<T>(v);
    }
  };
  if (p.chunks - (int)blockIdx.y * (64 * kEach) >= 64 * kEach) run(std::true_type());
  else run(std::false_type());
}

}  // namespace lpgemm
