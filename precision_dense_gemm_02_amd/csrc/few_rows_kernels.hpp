// Products of few rows with weights that are read once: 16-bit weights, or
// 4-bit ones with group scales.
#pragma once

#include "activation.hpp"
#include "few_rows_index.hpp"
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
  int x_lds_stride;         // XLDS: bytes of a row of X in LDS
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

// MT x 16 rows of X against NB x 16 rows of W per workgroup, whose waves take
// runs of blocks of 128 k in turn, with DEPTH of them in flight; their sums meet in LDS and are
// added in the waves' order.
//
// A lane loads 16 bytes of a weight row.  16-bit weights: 8 values of k, and
// four loads make a block.  4 bits: 32 values, a quarter of a block; the four
// lanes of a row exchange words, so that each K-step of 32 is one
// consecutive run (a group of 32 is then one step).
//
// 4 bits: the codes enter the matrix instruction as 24 + code (one or two
// operations per pair), the sum of x comes from a product with ones, and
//   C += scale * (sum x (24 + code) - (24 + zero) sum x)
// per group, in binary32.  The four lanes of a row load the scales of a block's
// groups and hand them round.
//
// Whole blocks need no check of k: a lane's offset stays, the descriptors'
// bases move.  Only the last run of an odd number of them takes its second
// block's lanes out of the scales' loads (few_rows_index.hpp): a mask of the
// offsets, 0.4% of the time of 120 products of 1 to 24 rows; records that end with
// the rows' scales, in scalar registers that some kernels do not have, 1.0%.
//
// Bound by the weights' stream with 16-bit weights (1 x 28672 x 4096 46 us, 5.1
// TB/s, the rate of a large copy).  With 4-bit ones the loads alone run at 4.4
// TB/s (1 x 14336 x 14336: 23.5 us of 30.9), the scales, 2 bytes from each of 16
// rows a load, add 4.5 us to them (groups of 64 with zeros 11), and the rest is
// the codes' way into the matrix instructions.  All of a segment's scales copied
// into LDS first: 16 x 14336 x 14336 43.0 -> 37.7 us, 1 x 4096 x 14336 11.6 ->
// 12.5, 16 x 14336 x 512 6.1 -> 8.7; X of 16 rows in LDS, 16 x
// 14336 x 4096: 18.4 -> 19.9; neither is kept.
//
// W4: 0 for 16-bit weights, else the K-steps of 32 that share a scale (1, 2,
// or 4 for groups of 128 and more).  XLDS: X, a few rows of it, is copied into
// LDS first, where its fragments cost no vector loads.
template <typename T, int W4, bool ZEROS, int MT, int NB, bool XLDS, int WAVES, int DEPTH>
__global__ __launch_bounds__(64 * WAVES) void few_rows(FewRowsArgs p) {
  static_assert(!XLDS || MT == 1, "a few rows");
  constexpr int kSub = W4 ? 4 / W4 : 1;                 // groups in a block
  constexpr int kLoads = W4 ? 1 : 4;                    // 16-byte loads per weight row and block
  constexpr int RUN = W4 ? kScaleRun : 1;               // consecutive blocks a wave takes: whole cache lines of a row
  constexpr int kScaleLoads = scale_loads(W4);          // per row and run, four groups each
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int m0 = blockIdx.y * (16 * MT);
  const bool gated = p.F > 0;
  const int per_half = gated ? NB / 2 : NB;   // column tiles of 16 per projection
  const int c0 = blockIdx.x * (16 * per_half);
  const int columns = gated ? p.F : p.N;
  const int blocks = (p.K + 127) >> 7, whole = p.K >> 7;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

  const int rows_x = min(16 * MT, p.M - m0);
  const uint8_t* const x_base = p.X + (size_t)m0 * p.x_stride;
  // a column tile's weight rows: the first, and how many
  auto first_row = [&](int nb) { return nb < per_half ? c0 + 16 * nb : p.F + c0 + 16 * (nb - per_half); };
  auto row_count = [&](int nb) { return max(min(columns - (c0 + 16 * (nb < per_half ? nb : nb - per_half)), 16), 0); };
  const uint8_t* w_base[NB];
  const uint8_t *s_base[NB], *z_base[NB];
  uint32_t w_off[NB], s_off[NB];              // this lane's, in block 0
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const size_t row = first_row(nb);
    w_base[nb] = p.W + row * p.row_bytes;
    s_base[nb] = (const uint8_t*)(p.scales + row * p.groups);
    z_base[nb] = (const uint8_t*)(p.zeros + row * p.groups);
    const bool row_here = r < row_count(nb);
    w_off[nb] = row_here ? (uint32_t)(r * p.row_bytes + 16 * q) : kOutOfRange;
    s_off[nb] = row_here ? 2u * (r * p.groups + scale_lane_group(W4, p.group_shift, q)) : kOutOfRange;
  }
  const uint32_t second_block = scale_second_block(W4, q) ? kOutOfRange : 0;
  uint32_t x_off[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) x_off[mt] = 16 * mt + r < rows_x ? (uint32_t)((16 * mt + r) * p.x_stride + 16 * q) : kOutOfRange;
  auto rsrc_of = [](const void* base, int bytes = 0x7FFFFFFF) { return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, bytes, kBufferWord3); };

  struct Run {
    i32x4 w[RUN][NB][kLoads];
    i32x4 x[XLDS ? 1 : RUN][MT][4];
    uint16_t s[NB][kScaleLoads], z[NB][kScaleLoads];   // of group q of the load
  };
  // a run of whole blocks, or (past the last) zeros: the loads go out in any
  // case, so that a wait on one leaves those behind it in flight
  const int runs = (whole + RUN - 1) / RUN;
  const int first_run = runs > 0 ? (int)(blockIdx.x * 5u % (uint32_t)runs) : 0;
  auto place = [&](int i) { const int run = i + first_run; return i >= runs ? whole : run >= runs ? run - runs : run; };
  auto load = [&](Run& b, int i) __attribute__((always_inline)) {
    const int run = place(i);
#pragma unroll
    for (int h = 0; h < RUN; ++h) {
      const int kb = run * RUN + h;
      const int bytes = kb < whole ? 0x7FFFFFFF : 0;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const auto rsrc = rsrc_of(w_base[nb] + (size_t)kb * (W4 ? 64 : 256), bytes);
#pragma unroll
        for (int l = 0; l < kLoads; ++l) b.w[h][nb][l] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, w_off[nb] + 64 * l, 0, 0);
      }
    }
    if constexpr (!XLDS) {
#pragma unroll
      for (int h = 0; h < RUN; ++h) {
        const int kb = run * RUN + h;
        const auto rsrc = rsrc_of(x_base + (size_t)kb * 256, kb < whole ? 0x7FFFFFFF : 0);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < 4; ++j) b.x[h][mt][j] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, x_off[mt] + 64 * j, 0, 0);
      }
    }
    if constexpr (W4 != 0) {
#pragma unroll
      for (int t = 0; t < kScaleLoads; ++t) {
        // groups of 32: those of block t of the run; of 64: two of each block; more: one of each (both may be the same)
        const int g = scale_first_group(W4, p.group_shift, run, t);
        const int bytes = scale_load_there(W4, run, t, whole) ? 0x7FFFFFFF : 0;
        const uint32_t not_there = W4 == 1 || run * RUN + 1 < whole ? 0 : second_block;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const uint32_t off = s_off[nb] | not_there;
          b.s[nb][t] = __builtin_amdgcn_raw_buffer_load_b16(rsrc_of(s_base[nb] + 2 * (size_t)g, bytes), off, 0, 0);
          b.z[nb][t] = ZEROS ? __builtin_amdgcn_raw_buffer_load_b16(rsrc_of(z_base[nb] + 2 * (size_t)g, bytes), off, 0, 0) : 0;
        }
      }
    }
  };
  // the last block, where the row ends inside it
  auto load_end = [&](Run& b) __attribute__((always_inline)) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        const int at = W4 ? whole * 64 : whole * 256 + 64 * l;
        b.w[0][nb][l] = __builtin_amdgcn_raw_buffer_load_b128(rsrc_of(w_base[nb]), at + 16 * q < p.row_bytes ? w_off[nb] + at : kOutOfRange, 0, 0);
      }
      if constexpr (W4 != 0) {
        const int g = W4 == 4 ? whole >> p.group_shift : whole * kSub;
        const int own = W4 == 4 ? 0 : W4 == 2 ? q & 1 : q;
        const uint32_t off = g + own < p.groups && w_off[nb] != kOutOfRange ? 2u * (r * p.groups + g + own) : kOutOfRange;
        b.s[nb][0] = __builtin_amdgcn_raw_buffer_load_b16(rsrc_of(s_base[nb]), off, 0, 0);
        b.z[nb][0] = ZEROS ? __builtin_amdgcn_raw_buffer_load_b16(rsrc_of(z_base[nb]), off, 0, 0) : 0;
      }
    }
    if constexpr (!XLDS) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = whole * 128 + 32 * j;
          b.x[0][mt][j] = __builtin_amdgcn_raw_buffer_load_b128(rsrc_of(x_base), at + 8 * q < p.K ? x_off[mt] + 2 * at : kOutOfRange, 0, 0);
        }
    }
  };

  f32x4 acc[MT][NB] = {};
  auto compute = [&](const Run& b, int h, int kb) __attribute__((always_inline)) {   // block h of the run
    i32x4 x[MT][4];
    if constexpr (XLDS) {
      const uint8_t* at = smem + min(r, rows_x - 1) * p.x_lds_stride + kb * 256 + 16 * q;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[0][j] = *(const i32x4*)(at + 64 * j);
    } else {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[mt][j] = W4 ? code_order(b.x[h][mt][j]) : b.x[h][mt][j];
    }
    if constexpr (W4 == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) acc[mt][nb] = mfma16<T>(x[mt][j], b.w[h][nb][j], acc[mt][nb]);
    } else {
      const int one = kIsF16<T> ? 0x3C003C00 : 0x3F803F80;
      const i32x4 ones = {one, one, one, one};
      u32x4 w[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) w[nb] = transpose_rows(__builtin_bit_cast(u32x4, b.w[h][nb][0]));
#pragma unroll
      for (int t = 0; t < kSub; ++t) {
        f32x4 sum[MT] = {}, part[MT][NB] = {};
#pragma unroll
        for (int j = t * W4; j < (t + 1) * W4; ++j) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) sum[mt] = mfma16<T>(x[mt][j], ones, sum[mt]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint32_t word = w[nb][j];
            const i32x4 f = code_fragment<T>(word);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) part[mt][nb] = mfma16<T>(x[mt][j], f, part[mt][nb]);
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int at = W4 == 1 ? h : 0, from = W4 == 1 ? t : W4 == 2 ? 2 * h + t : h;   // the load, and the lane row that holds the group
          const uint32_t sz = __shfl((int)(b.s[nb][at] | (uint32_t)b.z[nb][at] << 16), 16 * from + r);
          const float s = widen1<T>((uint16_t)sz), z = -kCodeBias - widen1<T>((uint16_t)(sz >> 16));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[mt][nb][e] = __builtin_fmaf(s, __builtin_fmaf(z, sum[mt][e], part[mt][nb][e]), acc[mt][nb][e]);
        }
      }
    }
  };

  {
    // X into LDS: rows of whole blocks, zeros behind K, in the order the
    // fragments need.  The first two chunks of each thread (with 8 waves 8192
    // values, with 4 waves 4096) are loaded before the weights and waited for
    // behind their loads; what is more, one row of 14336 for one, is copied in
    // front of both.
    const int chunks = blocks * 16;
    auto x_chunk = [&](int i) -> i32x4 {
      const int row = x_chunk_row(i, chunks), c = i - row * chunks;
      return i < rows_x * chunks && 8 * c < p.K ? *(const i32x4*)(x_base + (size_t)row * p.x_stride + 16 * c) : i32x4{0, 0, 0, 0};
    };
    auto put_chunk = [&](int i, const i32x4& v) {
      const int row = x_chunk_row(i, chunks), c = i - row * chunks;
      if (i < rows_x * chunks) *(i32x4*)(smem + row * p.x_lds_stride + 16 * c) = W4 ? code_order(v) : v;
    };
    const int threads = blockDim.x;
    i32x4 x0, x1;
    if constexpr (XLDS) {
      for (int i = 2 * threads + threadIdx.x; i < rows_x * chunks; i += threads) put_chunk(i, x_chunk(i));
      x0 = x_chunk(threadIdx.x);
      x1 = x_chunk(threads + threadIdx.x);
    }
    Run ring[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) load(ring[i], wave + i * waves);
    if constexpr (XLDS) {
      put_chunk(threadIdx.x, x0);
      put_chunk(threads + threadIdx.x, x1);
      __syncthreads();
    }
    for (int run = wave; run < runs; run += DEPTH * waves) {
#pragma unroll
      for (int i = 0; i < DEPTH; ++i) {
#pragma unroll
        for (int h = 0; h < RUN; ++h) {
          const int kb = place(run + i * waves) * RUN + h;
          if (kb < whole) compute(ring[i], h, kb);
        }
        load(ring[i], run + (i + DEPTH) * waves);
      }
    }
    if (whole < blocks && wave == runs % waves) {
      load_end(ring[0]);
      compute(ring[0], 0, whole);
    }
    if constexpr (XLDS) __syncthreads();
  }

  float* const red = (float*)smem;
  // sums: [wave][row][column], a column more for the banks
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
