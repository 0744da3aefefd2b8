// Products of few rows with weights that are read once: 16-bit weights, or
// 4-bit ones with group scales.
#pragma once

#include "activation.hpp"
#include "half_types.hpp"

namespace lpgemm {

struct FewRowsArgs {
  const uint8_t* X;         // M rows of K values
  const uint8_t* W;         // N rows of row_bytes (gated: the gate's F rows, then the up projection's)
  const uint16_t* scales;   // 4 bits: N x groups
  const uint16_t* zeros;    // ... or null
  uint8_t* C;               // M x N (gated: M x F)
  uint8_t* GU;              // gated: M x 2 F sums in the operands' type, or null
  int out_type;             // lpgemm_type of C
  int M, N, K;
  int F;                    // gated: N / 2, else 0
  int activation;
  int x_stride;             // bytes
  int row_bytes;            // of W
  int groups;               // scales of a row
  int group_shift;          // 4 bits, groups of 128 and more: log2 of a group's blocks
};

// Two codes of a word as values of T holding 24 + code, exactly: the nibble
// enters the mantissa of 16.0 below its top bit's place, which makes 16 + n for
// n = 0 .. 15, and the flipped sign bit turns two's complement into code + 8.
// Word pair `i`: codes i and i + 4 of the word.
template <typename T, int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  if constexpr (kIsF16<T>) {
    const uint32_t t = I == 0 ? w << 6 : I == 1 ? w << 2 : I == 2 ? w >> 2 : w >> 6;
    return (t & 0x03C003C0u) ^ 0x4E004E00u;
  } else {
    const uint32_t t = I == 0 ? w << 3 : I == 1 ? w >> 1 : I == 2 ? w >> 5 : w >> 9;
    return (t & 0x00780078u) ^ 0x41C041C0u;
  }
}
constexpr float kCodeBias = 24.f;

template <typename T>
__device__ __forceinline__ i32x4 code_fragment(uint32_t w) {
  return i32x4{(int)code_pair<T, 0>(w), (int)code_pair<T, 1>(w), (int)code_pair<T, 2>(w), (int)code_pair<T, 3>(w)};
}

// Eight consecutive values in the order of code_fragment: 0 4, 1 5, 2 6, 3 7.
__device__ __forceinline__ i32x4 code_order(const i32x4& x) {
  return i32x4{(int)__builtin_amdgcn_perm((uint32_t)x.z, (uint32_t)x.x, 0x05040100u),
               (int)__builtin_amdgcn_perm((uint32_t)x.z, (uint32_t)x.x, 0x07060302u),
               (int)__builtin_amdgcn_perm((uint32_t)x.w, (uint32_t)x.y, 0x05040100u),
               (int)__builtin_amdgcn_perm((uint32_t)x.w, (uint32_t)x.y, 0x07060302u)};
}

__device__ __forceinline__ void store_value(uint8_t* C, int out_type, size_t i, float v) {
  if (out_type == 0) ((float*)C)[i] = v;
  else ((uint16_t*)C)[i] = out_type == 1 ? narrow1<TypeF16>(v) : narrow1<TypeBF16>(v);
}

// The most wavefronts of a workgroup: registers bound it.
constexpr int few_rows_waves(int mt, int nb) { return mt * nb == 1 ? 16 : mt * nb == 8 ? 4 : 8; }

// MT x 16 rows of X against NB x 16 rows of W per workgroup, whose waves take
// the blocks of 128 k in turn; their sums meet in LDS and are added in the
// waves' order.
//
// A lane loads 16 bytes of a weight row.  16-bit weights: 8 values of k, and
// four loads make a block.  4 bits: 32 values, a quarter of a block; the four
// lanes of a row exchange words, so that each K-step of 32 is one
// consecutive run (a group of 32 is then one step).
//
// 4 bits: the codes enter the matrix instruction as 24 + code (one or two
// operations per pair), the sum of x comes from a product with ones, and
//   C += scale * (sum x (24 + code) - (24 + zero) sum x)
// per group, in binary32.
//
// W4: 0 for 16-bit weights, else the K-steps of 32 that share a scale (1, 2,
// or 4 for groups of 128 and more).
template <typename T, int W4, int MT, int NB>
__global__ __launch_bounds__(64 * few_rows_waves(MT, NB)) void few_rows(FewRowsArgs p) {
  constexpr int kSub = W4 ? 4 / W4 : 1;       // groups in a block
  constexpr int kLoads = W4 ? 1 : 4;          // 16-byte loads per weight row and block
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int m0 = blockIdx.y * (16 * MT);
  const bool gated = p.F > 0;
  const int per_half = gated ? NB / 2 : NB;   // column tiles of 16 per projection
  const int c0 = blockIdx.x * (16 * per_half);
  const int columns = gated ? p.F : p.N;
  const int blocks = (p.K + 127) >> 7;

  const int rows_x = min(16 * MT, p.M - m0);
  const auto rsrc_x = __builtin_amdgcn_make_buffer_rsrc((void*)(p.X + (size_t)m0 * p.x_stride), 0,
                                                        rows_x * p.x_stride, kBufferWord3);
  // first weight row of column tile nb, and how many there are
  auto first_row = [&](int nb) { return nb < per_half ? c0 + 16 * nb : p.F + c0 + 16 * (nb - per_half); };
  auto row_count = [&](int nb) { return max(min(columns - (c0 + 16 * (nb < per_half ? nb : nb - per_half)), 16), 0); };

  struct Block {
    i32x4 w[NB][kLoads];
    i32x4 x[MT][4];
    uint16_t s[NB][kSub], z[NB][kSub];
  };
  auto load = [&](Block& b, int kb) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = first_row(nb), count = row_count(nb);
      const auto rsrc_w = __builtin_amdgcn_make_buffer_rsrc((void*)(p.W + (size_t)row * p.row_bytes), 0,
                                                            count * p.row_bytes, kBufferWord3);
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        const int at = W4 ? kb * 64 + 16 * q : kb * 256 + 64 * l + 16 * q;
        b.w[nb][l] = __builtin_amdgcn_raw_buffer_load_b128(rsrc_w, at < p.row_bytes ? r * p.row_bytes + at : kOutOfRange, 0, 0);
      }
      if constexpr (W4 != 0) {
        const size_t g0 = (size_t)row * p.groups;
        const auto rsrc_s = __builtin_amdgcn_make_buffer_rsrc((void*)(p.scales + g0), 0, count * p.groups * 2, kBufferWord3);
        const auto rsrc_z = __builtin_amdgcn_make_buffer_rsrc((void*)(p.zeros ? p.zeros + g0 : p.scales), 0,
                                                              p.zeros ? count * p.groups * 2 : 0, kBufferWord3);
#pragma unroll
        for (int t = 0; t < kSub; ++t) {
          const int g = W4 == 4 ? kb >> p.group_shift : kb * kSub + t;
          const uint32_t off = g < p.groups ? 2 * (r * p.groups + g) : kOutOfRange;
          b.s[nb][t] = __builtin_amdgcn_raw_buffer_load_b16(rsrc_s, off, 0, 0);
          b.z[nb][t] = __builtin_amdgcn_raw_buffer_load_b16(rsrc_z, off, 0, 0);
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = kb * 128 + 32 * j + 8 * q;
        b.x[mt][j] = __builtin_amdgcn_raw_buffer_load_b128(rsrc_x, k < p.K ? (16 * mt + r) * p.x_stride + 2 * k : kOutOfRange, 0, 0);
      }
  };

  f32x4 acc[MT][NB] = {};
  auto compute = [&](const Block& b) {
    if constexpr (W4 == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) acc[mt][nb] = mfma16<T>(b.x[mt][j], b.w[nb][j], acc[mt][nb]);
    } else {
      const int one = kIsF16<T> ? 0x3C003C00 : 0x3F803F80;
      const i32x4 ones = {one, one, one, one};
      i32x4 x[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[mt][j] = code_order(b.x[mt][j]);
      u32x4 w[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) w[nb] = transpose_rows(__builtin_bit_cast(u32x4, b.w[nb][0]));
#pragma unroll
      for (int t = 0; t < kSub; ++t) {
        f32x4 sum[MT] = {}, part[MT][NB] = {};
#pragma unroll
        for (int j = t * W4; j < (t + 1) * W4; ++j) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) sum[mt] = mfma16<T>(x[mt][j], ones, sum[mt]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const i32x4 f = code_fragment<T>(w[nb][j]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) part[mt][nb] = mfma16<T>(x[mt][j], f, part[mt][nb]);
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float s = widen1<T>(b.s[nb][t]), z = -kCodeBias - widen1<T>(b.z[nb][t]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[mt][nb][e] = __builtin_fmaf(s, __builtin_fmaf(z, sum[mt][e], part[mt][nb][e]), acc[mt][nb][e]);
        }
      }
    }
  };

  if (wave < blocks) {
    Block b0, b1;
    load(b0, wave);
    int kb = wave;
    for (; kb + waves < blocks; kb += 2 * waves) {
      load(b1, kb + waves);
      compute(b0);
      load(b0, kb + 2 * waves);   // (past the end: zeros, unused)
      compute(b1);
    }
    if (kb < blocks) compute(b0);
  }

  // sums: [wave][row][column], a column more for the banks
  extern __shared__ __attribute__((aligned(16))) float red[];
  constexpr int kPitch = 16 * NB + 1, kWave = 16 * MT * kPitch;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave * kWave + (16 * mt + 4 * q + e) * kPitch + 16 * nb + r] = acc[mt][nb][e];
  __syncthreads();
  auto total = [&](int row, int column) {
    float v = 0.f;
    for (int w = 0; w < waves; ++w) v += red[w * kWave + row * kPitch + column];
    return v;
  };
  const int width = 16 * per_half;
  for (int i = threadIdx.x; i < rows_x * width; i += blockDim.x) {
    const int row = i / width, c = i - row * width;
    if (c0 + c >= columns) continue;
    const size_t at = (size_t)(m0 + row) * columns + c0 + c;
    float v = total(row, c);
    if (gated) {
      const float u = total(row, c + width);
      if (p.GU) {
        uint16_t* gu = (uint16_t*)p.GU + (size_t)(m0 + row) * p.N + c0 + c;
        gu[0] = narrow1<T>(v);
        gu[p.F] = narrow1<T>(u);
      }
      v = activate(v, p.activation) * u;
    }
    store_value(p.C, p.out_type, at, v);
  }
}

}  // namespace lpgemm
