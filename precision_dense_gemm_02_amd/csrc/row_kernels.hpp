// Row kernels of the quantised expert layer: residual + RMSNorm and
// silu(gate) * up with int8 rows, MXFP4 quantisation and its inverse.
//
// All of them are HBM-bound: every value is loaded once, sixteen bytes per
// lane, kept in registers through the reductions and written once.
#pragma once

#include "gemm_kernels.hpp"

namespace lpgemm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

struct TypeF16 {
  using x8 = f16x8;
  static constexpr bool kSquaresUnderflow = false;   // in binary32: the least is 2^-48
};
struct TypeBF16 {
  using x8 = bf16x8;
  static constexpr bool kSquaresUnderflow = true;
};

// A row whose largest magnitude is below this counts as zero: 127 (1 / a)
// then stays finite.
constexpr float kTinyRow = 0x1p-100f;
constexpr uint32_t kInfBits = 0x7F800000u;

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// |z| as bits: for finite values and infinities their order is that of the
// magnitudes, and every NaN lies above, so one integer maximum finds the
// largest magnitude and says whether the row holds anything non-finite.
__device__ __forceinline__ uint32_t magnitude_bits(float z) {
  return __builtin_bit_cast(uint32_t, z) & 0x7FFFFFFFu;
}

// Eight codes RNE(z inv) of values with |z inv| <= 127 (1 + 2^-22): adding
// 1.5 * 2^23 rounds the product to an integer and leaves its two's
// complement in the low byte of the sum.  The product is rounded to binary32
// before that, as the codes' definition says: no fused multiply-add here.
__device__ __forceinline__ uint64_t int8_codes(const f32x8& z, float inv) {
#pragma clang fp contract(off)
  uint32_t b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float product = z[e] * inv;
    const float rounded = product + 12582912.0f;
    b[e] = __builtin_bit_cast(uint32_t, rounded);
  }
  uint32_t w[2];
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * d + 1], b[4 * d], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * d + 3], b[4 * d + 2], 0x04000C0Cu);
    w[d] = lo | hi;
  }
  return (uint64_t)w[0] | ((uint64_t)w[1] << 32);
}

struct RowArgs {
  const uint8_t* X;
  const uint8_t* R;        // norm: may be null
  const uint8_t* weight;   // norm
  uint8_t* H;              // norm: may be null
  int8_t* Q;
  float* scale;
  int64_t x_stride, r_stride, h_stride;   // bytes
  int M, K;
  float eps;
};

// What a row kernel needs of its 8 values at chunk c (16 bytes of X): the
// norm's h = x + r (rounded to the type) or the activation's z.
//
// NORM: `h` keeps the chunk in the type (4 registers); z = h * weight is
// formed twice, for the maximum and for the codes.  Otherwise `z` is kept in
// binary32, as its exponential is dear.
template <typename T>
__device__ __forceinline__ f32x8 widen(const i32x4& v) {
  return __builtin_convertvector(__builtin_bit_cast(typename T::x8, v), f32x8);
}
template <typename T>
__device__ __forceinline__ i32x4 narrow(const f32x8& v) {
  return __builtin_bit_cast(i32x4, __builtin_convertvector(v, typename T::x8));
}
template <typename T>
__device__ __forceinline__ i32x4 add_rounded(const i32x4& x, const i32x4& r) {
  const f32x8 a = widen<T>(x), b = widen<T>(r);
  f32x8 s;
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = a[e] + b[e];
  return narrow<T>(s);
}
template <typename T>
__device__ __forceinline__ f32x8 weighted(const i32x4& h, const i32x4& w) {
  const f32x8 a = widen<T>(h), b = widen<T>(w);
  f32x8 z;
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = __fmul_rn(a[e], b[e]);   // exact: 11 (8) bits each
  return z;
}
// g / (1 + exp(-g)) * u, to within 8 units of 2^-24 (12 below g = -86).
// exp(-g) is 2^h (1 + l ln 2) with h the rounded -g log2(e) and l what the
// rounding and the constant left out: 2^h alone is off by |g| units (57 at g =
// -61).  The factor enters through the sum's multiply-add, and the sum is held
// as a quarter of 1 + exp(-g), whose reciprocal is a normal number up to where
// exp overflows (the reciprocal instruction flushes subnormal results: without
// the quarter every g below -87.3 gave 0).  Past that, at g = -88.72, the
// quotient is -0.  The clamp keeps h and l finite for every g (2^184 and 2^-184
// stand for all beyond).
//
// The instructions this adds to 2^h and a plain reciprocal are hidden where
// memory bounds the kernel (us, bfloat16 4096 x 14336 50.9 against 50.0, 2048 x
// 40000 111.9 against 112.7) and show where it does not (16 x 14336 4.4 against
// 4.0; 16384 x 1408, 69% of the lanes in use, 24.6 against 21.8).  The
// library's exponential and a division, good to 4 units, take 65 to 72, 143,
// 6.0 and 36.
template <typename T>
__device__ __forceinline__ f32x8 gated(const i32x4& gate, const i32x4& up) {
  const f32x8 g = widen<T>(gate), u = widen<T>(up);
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eRest = 0x1.4ae0cp-26f, kQuarterLn2 = 0x1.62e43p-3f;
  f32x8 z;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = -__builtin_amdgcn_fmed3f(g[e], -128.f, 128.f);
    const float h = __fmul_rn(x, kLog2e);
    const float l = __builtin_fmaf(x, kLog2eRest, __builtin_fmaf(x, kLog2e, -h));
    const float quarter = __builtin_fmaf(__builtin_amdgcn_exp2f(h), __builtin_fmaf(l, kQuarterLn2, 0.25f), 0.25f);
    z[e] = g[e] * (0.25f * __builtin_amdgcn_rcpf(quarter)) * u[e];
  }
  return z;
}

// Squares of h below 2^-63 are subnormal in binary32 or zero.  That shows in
// mean h^2 + eps only where both are small: then the sum is taken again, of
// h 2^100 (at most 2^10 2^-50 2^100 each, and at least 2^-133 2^100).  Rows of
// ordinary size pay a comparison (us with and without: 8192 x 8192 80.7, 80.5;
// 4096 x 32768 181.9, 180.2; one row of 4096 2.68, 2.64).
constexpr int kLift = 100;
constexpr float kLiftFactor = 0x1p100f;
__device__ __forceinline__ bool squares_underflow(float sumsq, const RowArgs& p) {
  return p.eps < 0x1p-100f && sumsq < (float)p.K * 0x1p-100f;
}

// The scale of a row and the factor of its codes, from the largest magnitude
// (as bits) and, for the norm, the sum of squares: of h, or of h 2^kLift.
template <bool NORM>
__device__ __forceinline__ void row_factors(uint32_t amax_bits, float sumsq, const RowArgs& p, float& scale,
                                            float& inv, bool lifted = false) {
  const float a = __builtin_bit_cast(float, amax_bits);
  inv = 0.f;
  if (amax_bits >= kInfBits || (NORM && !(sumsq < __builtin_inff()))) {
    scale = __builtin_nanf("");
  } else if (a < kTinyRow) {
    scale = 0.f;
  } else {
    inv = __fmul_rn(127.f, __fdiv_rn(1.f, a));
    scale = __fdiv_rn(a, 127.f);
    if (NORM) {
      const float eps = lifted ? p.eps * 0x1p100f * 0x1p100f : p.eps;
      const float rstd = __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sumsq, (float)p.K), eps)));
      if (lifted) {   // rstd is that of h 2^kLift; the exponents meet in integers
        scale = __builtin_amdgcn_ldexpf(__fmul_rn(__builtin_amdgcn_frexp_mantf(scale), rstd),
                                        __builtin_amdgcn_frexp_expf(scale) + kLift);
      } else {
        scale = __fmul_rn(scale, rstd);
      }
    }
  }
}

// Joins the waves of a row's workgroup: the largest bits and the sum.
template <int WPR, bool NORM>
__device__ __forceinline__ void row_join(uint32_t& amax, float& sumsq, int wave) {
  amax = wave_max_u32(amax);
  if (NORM) sumsq = wave_sum(sumsq);
  if constexpr (WPR > 1) {
    __shared__ uint32_t part_max[WPR];
    __shared__ float part_sum[WPR];
    if ((threadIdx.x & 63) == 0) {
      part_max[wave] = amax;
      part_sum[wave] = sumsq;
    }
    __syncthreads();
    amax = part_max[0];
    sumsq = part_sum[0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) {
      amax = max(amax, part_max[i]);
      sumsq += part_sum[i];
    }
  }
}

// Adds up the waves' second sums (in LDS of its own: the first may still be
// read).
template <int WPR>
__device__ __forceinline__ float row_sum_again(float sumsq, int wave) {
  sumsq = wave_sum(sumsq);
  if constexpr (WPR > 1) {
    __shared__ float part[WPR];
    if ((threadIdx.x & 63) == 0) part[wave] = sumsq;
    __syncthreads();
    sumsq = part[0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) sumsq += part[i];
  }
  return sumsq;
}
template <typename T>
__device__ __forceinline__ float lifted_squares(const i32x4& h, float sumsq) {
  const f32x8 f = widen<T>(h);
#pragma unroll
  for (int e = 0; e < 8; ++e) sumsq = __builtin_fmaf(f[e] * kLiftFactor, f[e] * kLiftFactor, sumsq);
  return sumsq;
}

// Rows of at most 512 WPR NC values, held in registers: WPR wavefronts share
// a row and each lane keeps its NC chunks of 8 values (chunk li + 64 WPR c).
// Chunks past the row's end load as zero through the buffer resource, which
// changes neither the maximum nor the sum of squares.  All loads of a row go
// out before the first is used: of one row with WPR > 1, of one per wave
// otherwise.
//
// Bound by HBM from a few hundred rows on (norm 7, activation 5 bytes a value;
// bfloat16, inputs in no cache: norm of 8192 x 8192 80.7 us, 5.8 TB/s; the
// activation of 4096 x 14336 50.9, 5.8 TB/s), below that by the launch and a
// trip to memory (1 x 4096 2.7 us, 16 x 14336 4.4).  Non-temporal stores would
// take 2 to 5% off the large ones and slow the product that reads the codes
// by more (activation of 4096 x 14336 and the product with 4096 columns 249
// against 234 us; 1024 rows 116 against 118).
template <typename T, bool NORM, int WPR, int NC>
__global__ __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) void rows_int8_regs(RowArgs p) {
  constexpr int kRowLanes = 64 * WPR;
  constexpr int kRowsPerGroup = WPR == 1 ? 4 : 1;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = blockIdx.x * kRowsPerGroup + (WPR == 1 ? wave : 0);
  const int li = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  if (WPR == 1 && row >= p.M) return;   // with WPR > 1 the grid has exactly M workgroups
  const int chunks = p.K >> 3;
  auto rsrc = [&](const uint8_t* base, int64_t stride, int64_t skip) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)(base + row * stride + skip), 0, p.K * 2, kBufferWord3);
  };
  const __amdgpu_buffer_rsrc_t rx = rsrc(p.X, p.x_stride, 0);
  // norm: the residual (empty when absent); activation: the up half
  const __amdgpu_buffer_rsrc_t ry =
      NORM ? __builtin_amdgcn_make_buffer_rsrc((void*)(p.R ? p.R + row * p.r_stride : p.X), 0, p.R ? p.K * 2 : 0,
                                               kBufferWord3)
           : rsrc(p.X, p.x_stride, (int64_t)p.K * 2);
  const __amdgpu_buffer_rsrc_t rw =
      __builtin_amdgcn_make_buffer_rsrc((void*)p.weight, 0, NORM ? p.K * 2 : 0, kBufferWord3);

  i32x4 x[NC], y[NC], w[NORM ? NC : 1];
#pragma unroll
  for (int c = 0; c < NC; ++c) x[c] = __builtin_amdgcn_raw_buffer_load_b128(rx, (li + kRowLanes * c) * 16, 0, 0);
#pragma unroll
  for (int c = 0; c < NC; ++c) y[c] = __builtin_amdgcn_raw_buffer_load_b128(ry, (li + kRowLanes * c) * 16, 0, 0);
  if constexpr (NORM) {
#pragma unroll
    for (int c = 0; c < NC; ++c) w[c] = __builtin_amdgcn_raw_buffer_load_b128(rw, (li + kRowLanes * c) * 16, 0, 0);
  }

  uint32_t amax = 0;
  float sumsq = 0.f;
  f32x8 zs[NORM ? 1 : NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    f32x8 z;
    if constexpr (NORM) {
      if (p.R) x[c] = add_rounded<T>(x[c], y[c]);
      const int idx = li + kRowLanes * c;
      if (p.H && idx < chunks) *(i32x4*)(p.H + row * p.h_stride + (int64_t)idx * 16) = x[c];
      const f32x8 h = widen<T>(x[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) sumsq = __builtin_fmaf(h[e], h[e], sumsq);
      z = weighted<T>(x[c], w[c]);
    } else {
      z = gated<T>(x[c], y[c]);
      zs[c] = z;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max(amax, magnitude_bits(z[e]));
  }
  row_join<WPR, NORM>(amax, sumsq, wave);
  bool lifted = false;
  if constexpr (NORM && T::kSquaresUnderflow) {
    lifted = squares_underflow(sumsq, p);   // one answer for the row's lanes
    if (lifted) {
      sumsq = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) sumsq = lifted_squares<T>(x[c], sumsq);
      sumsq = row_sum_again<WPR>(sumsq, wave);
    }
  }
  float scale, inv;
  row_factors<NORM>(amax, sumsq, p, scale, inv, lifted);
  if (li == 0) p.scale[row] = scale;
  uint64_t* const q = (uint64_t*)(p.Q + (int64_t)row * p.K);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int idx = li + kRowLanes * c;
    if (idx < chunks) {
      if constexpr (NORM) q[idx] = inv != 0.f ? int8_codes(weighted<T>(x[c], w[c]), inv) : 0;
      else q[idx] = inv != 0.f ? int8_codes(zs[c], inv) : 0;
    }
  }
}

// Longer rows (and K = 0): a workgroup per row and two passes over it, the
// second mostly from the L2 (us, norm of 2048 x 40000 131, 4.4 TB/s; activation
// of 2048 x 40000 112, 3.7 TB/s, its exponentials twice).  A thread handles the same chunks in all, so
// a later one may read back an H that overwrote X or R.
template <typename T, bool NORM>
__global__ __launch_bounds__(1024) void rows_int8_long(RowArgs p) {
  const int row = blockIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int chunks = p.K >> 3;
  const i32x4* const x = (const i32x4*)(p.X + row * p.x_stride);
  const i32x4* const r = p.R ? (const i32x4*)(p.R + row * p.r_stride) : nullptr;
  const i32x4* const w = (const i32x4*)p.weight;
  i32x4* const h = p.H ? (i32x4*)(p.H + row * p.h_stride) : nullptr;
  uint32_t amax = 0;
  float sumsq = 0.f;
  for (int c = threadIdx.x; c < chunks; c += 1024) {
    f32x8 z;
    if constexpr (NORM) {
      const i32x4 v = r ? add_rounded<T>(x[c], r[c]) : x[c];
      if (h) h[c] = v;
      const f32x8 f = widen<T>(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sumsq = __builtin_fmaf(f[e], f[e], sumsq);
      z = weighted<T>(v, w[c]);
    } else {
      z = gated<T>(x[c], x[c + chunks]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max(amax, magnitude_bits(z[e]));
  }
  row_join<16, NORM>(amax, sumsq, wave);
  // the row's h in the passes after the first: an H that overwrote X or R is
  // read back
  auto h_again = [&](int c) { return h ? h[c] : (r ? add_rounded<T>(x[c], r[c]) : x[c]); };
  bool lifted = false;
  if constexpr (NORM && T::kSquaresUnderflow) {
    lifted = squares_underflow(sumsq, p);   // one answer for the row's lanes
    if (lifted) {
      sumsq = 0.f;
      for (int c = threadIdx.x; c < chunks; c += 1024) sumsq = lifted_squares<T>(h_again(c), sumsq);
      sumsq = row_sum_again<16>(sumsq, wave);
    }
  }
  float scale, inv;
  row_factors<NORM>(amax, sumsq, p, scale, inv, lifted);
  if (threadIdx.x == 0) p.scale[row] = scale;
  uint64_t* const q = (uint64_t*)(p.Q + (int64_t)row * p.K);
  for (int c = threadIdx.x; c < chunks; c += 1024) {
    f32x8 z;
    if constexpr (NORM) z = weighted<T>(h_again(c), w[c]);
    else z = gated<T>(x[c], x[c + chunks]);
    q[c] = inv != 0.f ? int8_codes(z, inv) : 0;
  }
}

// ---------------------------------------------------------------------------
// MXFP4.  Four lanes share a block of 32 values, eight each; the largest
// magnitude's exponent field E (of its binary32 form) gives the scale byte
// b = clamp(E - 2, 0, 254), since floor(log2 a) = E - 127 for a normal a and
// anything smaller clamps to 0.  The conversion instruction divides by
// 2^(b - 127), rounds to nearest even and saturates at 6.
struct Mxfp4Args {
  const uint8_t* X;
  uint8_t* codes;
  uint8_t* scales;
  int64_t x_stride;      // bytes
  int chunks;            // K / 8
  int scale_stride;
  uint32_t total;        // rows x chunks of this launch
};

// One block of a row by the four lanes that hold its values v, at chunk c.
template <typename T>
__device__ __forceinline__ void quantize_chunk(const Mxfp4Args& p, i32x4 v, uint32_t row, uint32_t c, bool on) {
  f32x8 x = widen<T>(v);
  uint32_t amax = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = max(amax, magnitude_bits(x[e]));
  amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1));
  amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2));
  const int field = (int)(amax >> 23);
  const int b = field == 255 ? 255 : max(field - 2, 0);
  // blocks of very small values are scaled up first, so that the divisor
  // stays a normal number
  const bool small = b < 64;
  if (small) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= 0x1p64f;
  }
  const float unit = __builtin_bit_cast(float, (uint32_t)(small ? b + 64 : b) << 23);
  uint32_t code = 0;
  if (b != 255) {
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, x[0], x[1], unit, 0);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, x[2], x[3], unit, 1);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, x[4], x[5], unit, 2);
    code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, x[6], x[7], unit, 3);
  }
  if (!on) return;
  *(uint32_t*)(p.codes + (int64_t)row * p.chunks * 4 + (int64_t)c * 4) = code;
  if ((c & 3) == 0) {
    uint8_t* const s = p.scales + (int64_t)row * p.scale_stride;
    s[c >> 2] = (uint8_t)b;
    if (c + 4 == (uint32_t)p.chunks)
      for (int i = (p.chunks >> 2); i < p.scale_stride; ++i) s[i] = 0;
  }
}

// UNROLL chunks per lane, 256 apart, all loaded before the first is used.
// HBM-bound: 2 + 17/32 bytes a value (bfloat16, inputs in no cache: 14336 x
// 4096 29.8 us, 5.0 TB/s; 33 x 4096 2.0).  Non-temporal loads: 97 against 104
// at 32768 x 7168, but 36.1 against 35.6 at 8192 x 4096 where the values were
// just written.
template <typename T, int UNROLL>
__global__ __launch_bounds__(256) void quantize_mxfp4_kernel(Mxfp4Args p) {
  i32x4 v[UNROLL];
  uint32_t row[UNROLL], c[UNROLL];
  bool on[UNROLL];   // a block's four lanes are on together: chunks is a multiple of 4
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const uint32_t idx = (blockIdx.x * UNROLL + u) * 256u + threadIdx.x;
    on[u] = idx < p.total;
    row[u] = on[u] ? idx / (uint32_t)p.chunks : 0;
    c[u] = on[u] ? idx - row[u] * (uint32_t)p.chunks : 0;
    v[u] = i32x4{0, 0, 0, 0};
    if (on[u]) v[u] = *(const i32x4*)(p.X + (int64_t)row[u] * p.x_stride + (int64_t)c[u] * 16);
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) quantize_chunk<T>(p, v[u], row[u], c[u], on[u]);
}

// Eight values per lane and chunk: code times 2^(b - 127), in binary32, rounded
// to the output's type (OUT: 0 binary32, 1 binary16, 2 bfloat16); UNROLL
// chunks, 256 apart.  Bound by its stores (to bfloat16, 14336 x 4096, in no cache: 29.8 us, 5.0 TB/s).
// Non-temporal ones are faster alone (4096 x 4096 9.4 against 10.5 us) and
// slow down whoever reads the values next (with a product of 64 rows behind
// it 35.1 against 31.9).
struct Dequant4Args {
  const uint8_t* codes;
  const uint8_t* scales;
  uint8_t* Y;
  int chunks;
  int scale_stride;
  uint32_t total;
};

template <int OUT, int UNROLL>
__global__ __launch_bounds__(256) void dequantize_mxfp4_kernel(Dequant4Args p) {
  uint32_t codes[UNROLL], bytes[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const uint32_t idx = (blockIdx.x * UNROLL + u) * 256u + threadIdx.x;
    codes[u] = bytes[u] = 0;
    if (idx < p.total) {
      const uint32_t row = idx / (uint32_t)p.chunks, c = idx - row * (uint32_t)p.chunks;
      codes[u] = *(const uint32_t*)(p.codes + (int64_t)idx * 4);
      bytes[u] = p.scales[(int64_t)row * p.scale_stride + (c >> 2)];
    }
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const uint32_t idx = (blockIdx.x * UNROLL + u) * 256u + threadIdx.x;
    if (idx >= p.total) return;
    const uint32_t code = codes[u], b = bytes[u];
    // 2^(b - 127); b = 0 is a subnormal, 255 a NaN
    const float unit = __builtin_bit_cast(float, b == 255 ? 0x7FC00000u : (b == 0 ? 0x00400000u : b << 23));
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const f32x2_t v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.f, 0);
    const f32x2_t v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.f, 1);
    const f32x2_t v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.f, 2);
    const f32x2_t v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.f, 3);
    f32x8 y = {v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= unit;
    if constexpr (OUT == 0) {
      f32x8* const out = (f32x8*)(p.Y + (int64_t)idx * 32);
      *out = y;
    } else if constexpr (OUT == 1) {
      *(i32x4*)(p.Y + (int64_t)idx * 16) = narrow<TypeF16>(y);
    } else {
      *(i32x4*)(p.Y + (int64_t)idx * 16) = narrow<TypeBF16>(y);
    }
  }
}

}  // namespace lpgemm
