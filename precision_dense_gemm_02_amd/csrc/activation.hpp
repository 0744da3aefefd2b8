// The activations of a gated block and their derivatives, in binary32.
#pragma once

#include <hip/hip_runtime.h>

namespace lpgemm {

// (as lpgemm_activation)
constexpr int kSilu = 0, kGelu = 1;

// 1 / (1 + exp(-a)), to within 8 units of 2^-24 (12 below a = -86).  exp(-a)
// is 2^h (1 + l ln 2) with h the rounded -a log2(e) and l what the rounding
// and the constant left out; the sum is held as a quarter of 1 + exp(-a), so
// that its reciprocal is a normal number up to where exp overflows (a =
// -88.72, 0 from there on).  A NaN gives some value between 0 and 1: every use
// multiplies by a NaN as well.
__device__ __forceinline__ float logistic(float a) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eRest = 0x1.4ae0cp-26f, kQuarterLn2 = 0x1.62e43p-3f;
  const float x = -__builtin_amdgcn_fmed3f(a, -128.f, 128.f);
  const float h = __fmul_rn(x, kLog2e);
  const float l = __builtin_fmaf(x, kLog2eRest, __builtin_fmaf(x, kLog2e, -h));
  const float quarter = __builtin_fmaf(__builtin_amdgcn_exp2f(h), __builtin_fmaf(l, kQuarterLn2, 0.25f), 0.25f);
  return 0.25f * __builtin_amdgcn_rcpf(quarter);
}

// GELU in its tanh form is g times the logistic function of
// 2 sqrt(2 / pi) (g + 0.044715 g^3).
constexpr float kGelu1 = 1.5957691216057308f;                // 2 sqrt(2 / pi)
constexpr float kGelu3 = 1.5957691216057308f * 0.044715f;

__device__ __forceinline__ float gelu_argument(float g) { return g * __builtin_fmaf(kGelu3, g * g, kGelu1); }

__device__ __forceinline__ float activate(float g, int kind) {
  return g * logistic(kind == kSilu ? g : gelu_argument(g));
}

// act(g) and act'(g), for results that are rounded to 16 bits.  With p =
// logistic(a(g)): act = g p, act' = p + g a' p (1 - p).  p and 1 - p are 1 / (1 +
// e) and e / (1 + e) with e = exp(-|a|), which neither cancels nor overflows.
// The exponential is one instruction, off by |a| units of 2^-24: at most 2^-17
// of the value, and 0 past |a| = 87.3, where it would be subnormal.  Past |g| = 16 the second term of GELU's derivative is below
// 2^-140; clamped there, g^2 a' stays finite.
__device__ __forceinline__ void activate_with_slope(float g, int kind, float& act, float& slope) {
  const float a = kind == kSilu ? g : gelu_argument(g);
  const float e = __builtin_amdgcn_exp2f(-1.442695041f * __builtin_fabsf(a));
  const float more = __builtin_amdgcn_rcpf(1.f + e), less = e * more;
  const float p = a < 0.f ? less : more, rest = a < 0.f ? more : less;
  act = g * p;
  if (kind == kSilu) {
    slope = __builtin_fmaf(act, rest, p);
  } else {
    const float gc = __builtin_amdgcn_fmed3f(g, -16.f, 16.f);
    slope = __builtin_fmaf(gc * __builtin_fmaf(3.f * kGelu3, gc * gc, kGelu1) * rest, p, p);
  }
}

}  // namespace lpgemm
