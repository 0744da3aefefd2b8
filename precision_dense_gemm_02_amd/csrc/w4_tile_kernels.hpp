// Products of many rows with 4-bit weights that have group scales.
#pragma once

#include "few_rows_kernels.hpp"

namespace lpgemm {

struct W4TileArgs {
  const uint8_t* X;         // M rows of K values
  const uint8_t* W;         // N rows of row_bytes (gated: the gate's F rows, then the up projection's)
  const uint16_t* scales;   // N x groups
  const uint16_t* zeros;    // ... or null
  uint8_t* C;               // M x N (gated: M x F)
  float* part;              // splits > 1: splits x M x N sums
  int out_type;             // lpgemm_type of C
  int M, N, K;
  int F;                    // gated: N / 2, else 0
  int activation;
  int x_stride;             // bytes
  int row_bytes;            // of W
  int groups;               // of a row
  int group_shift;          // log2 of a group's values
  int stages;               // of 128 k, all of them
  int split_stages;         // ... of one split (blockIdx.y)
  int splits;
  int tiles_m, tiles_n;
};

// Two bytes per lane, zero-extended: lane l's word lands at lds_addr + 4 l.
__device__ __forceinline__ void lds_dma_2(const i32x4& rsrc, uint32_t lds_addr, uint32_t voff) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "buffer_load_ushort %2, %3, 0 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "s"(lds_addr), "v"(voff), "s"(rsrc)
      : "memory");
}

// Two consecutive codes of a byte as values of T holding 24 + code (see
// code_pair), in their own order: byte `I` goes to the upper byte of both
// halves, and each half is shifted to where its nibble enters the mantissa.
template <typename T, int I>
__device__ __forceinline__ uint32_t code_pair_in_order(uint32_t w) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  constexpr uint32_t kSel = 0x000C000Cu | ((uint32_t)I << 8) | ((uint32_t)I << 24);
  const u16x2 b = __builtin_bit_cast(u16x2, __builtin_amdgcn_perm(0u, w, kSel));
  if constexpr (kIsF16<T>) {   // nibbles from bits 8 and 12 to bit 6
    const u16x2 t = b >> u16x2{2, 6};
    return (__builtin_bit_cast(uint32_t, t) & 0x03C003C0u) ^ 0x4E004E00u;
  } else {                     // ... to bit 3
    const u16x2 t = b >> u16x2{5, 9};
    return (__builtin_bit_cast(uint32_t, t) & 0x00780078u) ^ 0x41C041C0u;
  }
}
template <typename T>
__device__ __forceinline__ i32x4 code_fragment_in_order(uint32_t w) {
  return i32x4{(int)code_pair_in_order<T, 0>(w), (int)code_pair_in_order<T, 1>(w), (int)code_pair_in_order<T, 2>(w),
               (int)code_pair_in_order<T, 3>(w)};
}

// The splits' sums added in order.
template <typename T>
__global__ __launch_bounds__(256) void join_w4(W4TileArgs p) {
  const int columns = p.F > 0 ? p.F : p.N;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int row = (int)(i / columns), col = (int)(i - (int64_t)row * columns);
  if (row >= p.M) return;
  float v = 0.f, u = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float* part = p.part + ((size_t)s * p.M + row) * p.N + col;
    v += part[0];
    if (p.F > 0) u += part[p.F];
  }
  store_value(p.C, p.out_type, i, p.F > 0 ? activate(v, p.activation) * u : v);
}

// Tiles of BM rows by 128 columns, 32 of them for each of four waves, and a
// ring of STAGES K-stages of 128: X's rows (256 bytes), the weights' rows (64
// bytes of codes), and each wave's own scales and zeros, all by direct-to-LDS
// loads.  Lane l has k = 32 g + 16 (l / 32) + 8 b .. + 7 of the stage in K-step
// 2 g + b: a group of 32 is two steps, a weight row's two steps are 8 bytes.
//
// The codes enter the matrix instructions as 24 + code, exactly, the sums of x
// come from a product with ones, and
//   C += scale * (sum x (24 + code) - (24 + zero) sum x)
// per group, in binary32.
//
// WK groups of four waves take the stages in turn, each through a ring of its
// own, and add their sums in LDS at the end: wavefronts to switch to while
// another waits for LDS, without more tiles or splits.
//
// Bound by the codes' conversion and by LDS latency, not by memory: 32 x 14336 x
// 4096 bf16, groups of 64 with zeros 21.0 us (1.6 TB/s; with WK = 2 22.3, with one
// group of four waves 24.4).
//
// STEPS: K-steps of 32 that share a scale (1, 2, or 4 for groups of 128 and more).
template <typename T, int STEPS, int BM, int STAGES, int WK, bool GATED>
__global__ __launch_bounds__(256 * WK) void w4_tile(W4TileArgs p) {
  constexpr int BN = 128, TM = BM / 32;
  constexpr int kGroups = 4 / STEPS;                           // of a stage
  constexpr int kA = BM * 256, kB = BN * 64;
  constexpr int kScLoads = (kGroups * 32 + 63) / 64;           // of scales, and of zeros, per wave and stage
  constexpr int kWave = 2 * kScLoads * 256;                    // a wave's own bytes of a stage
  constexpr int kStage = kA + kB + 4 * kWave;
  constexpr int kSlotsA = BM / 16, kSlotsB = BN / 64;          // 1 KiB loads per wave and stage
  constexpr int kLoads = kSlotsA + kSlotsB + 2 * kScLoads;
  constexpr int kInFlight = (STAGES - 2) * kLoads;
  static_assert(kInFlight + kLoads <= 63, "vmcnt range");
  constexpr int kPitch = BN + 1;                               // of the staged sums
  constexpr int kEpi = BM * kPitch * 4;                        // one group's
  constexpr int kRing = STAGES * kStage > kEpi ? STAGES * kStage : kEpi;
  constexpr int kLds = WK * kRing;
  static_assert(kLds <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kLds];

  const int lane = threadIdx.x & 63;
  const int wk = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3), wn = wave;   // of the group
  const int logical = xcd_logical(blockIdx.x, p.tiles_m * p.tiles_n);
  const int band = logical / (8 * p.tiles_n), in_band = logical - band * 8 * p.tiles_n;
  const int height = min(p.tiles_m - 8 * band, 8);
  const int m0 = (8 * band + in_band % height) * BM;
  constexpr int kTileColumns = GATED ? BN / 2 : BN;
  const int c0 = (in_band / height) * kTileColumns;
  const int columns = GATED ? p.F : p.N;
  const int rows = min(BM, p.M - m0), cols = min(kTileColumns, columns - c0);
  const int s_begin = blockIdx.y * p.split_stages, s_end = min(s_begin + p.split_stages, p.stages);

  uint8_t* const ring = smem + wk * kRing;
  const uint32_t ring_lds = lds_address(ring);
  const i32x4 rsrc_x = make_rsrc(p.X + (size_t)m0 * p.x_stride, (uint32_t)rows * p.x_stride);
  // weight row (and scales' row) of the tile's column c: gate columns first
  auto weight_row = [&](int c) { return GATED && c >= BN / 2 ? p.F + c0 + c - BN / 2 : c0 + c; };
  auto column_here = [&](int c) { return (GATED && c >= BN / 2 ? c - BN / 2 : c) < cols; };

  uint32_t x_off[kSlotsA], x_col, w_off[kSlotsB], w_col;
  {
    const int r = 4 * wave + lane / 16;                         // (rows 16 apart have the same swizzle)
    x_col = RowLayout<256>::pos(r, lane % 16) * 16;
#pragma unroll
    for (int t = 0; t < kSlotsA; ++t) x_off[t] = (uint32_t)(16 * t + r) * p.x_stride + x_col;
    const int c = 16 * wave + lane / 4;                         // (rows 64 apart have the same swizzle)
    w_col = RowLayout<64>::pos(c, lane % 4) * 16;
#pragma unroll
    for (int t = 0; t < kSlotsB; ++t)
      w_off[t] = column_here(64 * t + c) ? (uint32_t)(64 * t + c - (GATED && 64 * t + c >= BN / 2 ? BN / 2 : 0)) * p.row_bytes + w_col : kOutOfRange;
  }
  const i32x4 rsrc_w = make_rsrc(p.W + (size_t)c0 * p.row_bytes, (uint32_t)cols * p.row_bytes);
  const i32x4 rsrc_up = make_rsrc(p.W + (size_t)(GATED ? p.F + c0 : c0) * p.row_bytes, (uint32_t)cols * p.row_bytes);
  // scales of this wave's columns: lane l of load t has column l % 32, group 2 t + l / 32 of the stage
  const bool wave_up = GATED && wn * 32 >= BN / 2;             // (a wave's columns are of one projection)
  const int wave_row0 = weight_row(wn * 32);
  const int wave_cols = max(min(cols - (wn * 32 - (wave_up ? BN / 2 : 0)), 32), 0);
  const i32x4 rsrc_s = make_rsrc(p.scales + (size_t)wave_row0 * p.groups, (uint32_t)wave_cols * p.groups * 2);
  const i32x4 rsrc_z = make_rsrc(p.zeros ? p.zeros + (size_t)wave_row0 * p.groups : p.scales, p.zeros ? (uint32_t)wave_cols * p.groups * 2 : 0);
  const uint32_t s_off = 2u * ((uint32_t)(lane % 32) * p.groups + lane / 32);
  // the group's i-th stage
  auto issue_stage = [&](int i, int at) __attribute__((always_inline)) {
    const int s = s_begin + i * WK + wk;
    const uint32_t slot = ring_lds + at * kStage;
    const bool live = s < s_end;
    const uint32_t kx = (uint32_t)s * 256, kw = (uint32_t)s * 64;
#pragma unroll
    for (int t = 0; t < kSlotsA; ++t)
      lds_dma_16(rsrc_x, slot + (4 * t + wave) * 1024, live && kx + x_col < 2u * p.K ? x_off[t] + kx : kOutOfRange);
#pragma unroll
    for (int t = 0; t < kSlotsB; ++t) {
      const uint32_t from = live && kw + w_col < (uint32_t)p.row_bytes && w_off[t] != kOutOfRange ? w_off[t] + kw : kOutOfRange;
      if (GATED && 64 * t >= BN / 2) lds_dma_16(rsrc_up, slot + kA + (4 * t + wave) * 1024, from);
      else lds_dma_16(rsrc_w, slot + kA + (4 * t + wave) * 1024, from);
    }
    const uint32_t own = slot + kA + kB + wave * kWave;
    const int g0 = (s * 128) >> p.group_shift;                  // (a group of 256 is that of two stages)
#pragma unroll
    for (int t = 0; t < kScLoads; ++t) {
      const int g = 2 * t + lane / 32;
      const uint32_t from = live && g < kGroups && g0 + g < p.groups ? s_off + 2 * (g0 + 2 * t) : kOutOfRange;
      lds_dma_2(rsrc_s, own + t * 256, from);
      lds_dma_2(rsrc_z, own + (kScLoads + t) * 256, from);
    }
  };

  const int fr = lane & 31, fh = lane >> 5;
  f32x16 acc[TM] = {};
  const int one = kIsF16<T> ? 0x3C003C00 : 0x3F803F80;
  const i32x4 ones = {one, one, one, one};

  const int rounds = (s_end - s_begin + WK - 1) / WK;   // (stages past the last are zeros)
  if (rounds > 0) {
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue_stage(i, i);
    int at = 0;
    for (int i = 0; i < rounds; ++i) {
      wait_vmcnt<kInFlight>();   // own loads of the stage landed
      wait_lgkmcnt0();           // own reads of the stage before done
      block_barrier();           // ... everyone's
      issue_stage(i + STAGES - 1, at == 0 ? STAGES - 1 : at - 1);
      const uint8_t* const slot = ring + at * kStage;
      const uint8_t* const own = slot + kA + kB + wave * kWave;
      at = at == STAGES - 1 ? 0 : at + 1;
      // everything the stage needs from LDS, before the first product
      float scale[kGroups], bias[kGroups];
      u32x2 code[4];
      i32x4 a[TM][8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        code[q] = *(const u32x2*)(slot + kA + RowLayout<64>::off(wn * 32 + fr, q) + 8 * fh);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int b = 0; b < 2; ++b) a[i][2 * q + b] = *(const i32x4*)(slot + RowLayout<256>::off(32 * i + fr, 4 * q + 2 * fh + b));
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int at = (g * 32 + fr) * 4;
        scale[g] = widen1<T>(*(const uint16_t*)(own + at));
        bias[g] = -kCodeBias - widen1<T>(*(const uint16_t*)(own + kScLoads * 256 + at));
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        f32x16 part[TM] = {}, sum[TM] = {};
#pragma unroll
        for (int q = g * STEPS; q < (g + 1) * STEPS; ++q)      // 32 values of k
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const uint32_t word = b ? code[q].y : code[q].x;
            const i32x4 f = code_fragment_in_order<T>(word);
#pragma unroll
            for (int i = 0; i < TM; ++i) {
              part[i] = mfma32<T>(a[i][2 * q + b], f, part[i]);
              sum[i] = mfma32<T>(a[i][2 * q + b], ones, sum[i]);
            }
          }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            acc[i][e] = __builtin_fmaf(scale[g], __builtin_fmaf(bias[g], sum[i][e], part[i][e]), acc[i][e]);
      }
    }
  }

  // the sums through LDS
  wait_vmcnt<0>();
  wait_lgkmcnt0();
  block_barrier();
  {
    float* const staged = (float*)ring;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) staged[(32 * i + 8 * (e >> 2) + 4 * fh + (e & 3)) * kPitch + 32 * wn + fr] = acc[i][e];
    __syncthreads();
    auto total = [&](int r, int c) {   // the groups' sums, in order
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < WK; ++w) v += ((const float*)(smem + w * kRing))[r * kPitch + c];
      return v;
    };
    for (int i = threadIdx.x; i < rows * kTileColumns; i += 256 * WK) {
      const int r = i / kTileColumns, c = i % kTileColumns;
      if (c >= cols) continue;
      const size_t row = m0 + r;
      float v = total(r, c);
      if (p.splits > 1) {
        float* part = p.part + ((size_t)blockIdx.y * p.M + row) * p.N + c0 + c;
        part[0] = v;
        if constexpr (GATED) part[p.F] = total(r, BN / 2 + c);
      } else {
        if constexpr (GATED) v = activate(v, p.activation) * total(r, BN / 2 + c);
        store_value(p.C, p.out_type, row * columns + c0 + c, v);
      }
    }
  }
}

}  // namespace lpgemm
