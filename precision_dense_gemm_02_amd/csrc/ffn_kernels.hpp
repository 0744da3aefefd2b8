// The products of the gated feed-forward block and of its gradients, on 16-bit
// operands:
//
//   C = A . B   M x N over K,   A(m, k), B(k, n)
//
// Either operand may lie along k (rows of K values, as activations and
// weights do in the forward pass) or across it (K rows of M or N values: the
// gradients read the same arrays the other way).
#pragma once

#include <utility>

#include "activation.hpp"
#include "few_rows_kernels.hpp"

namespace lpgemm {

// What becomes of a tile of sums.
enum TileEnd {
  END_STORE = 0,       // C, in out_type
  END_GATED = 1,       // columns are pairs gate, up: H = act(gate) * up in out_type, and [gate up] if GU is set
  END_GATED_GRAD = 2,  // sums are dh: from [gate up] in GU, [dg du] into DGU and h into H
};

struct TileArgs {
  const uint8_t* A;
  const uint8_t* B;        // END_GATED: the gate's rows, then F rows of the up projection
  int64_t a_stride;        // bytes from one stored row to the next
  int64_t b_stride;
  uint8_t* C;              // END_STORE: rows of N values
  int out_type;            // lpgemm_type of C (END_GATED: of H)
  uint8_t* H;              // M x F
  uint8_t* GU;             // M x 2 F
  uint8_t* DGU;            // M x 2 F
  int activation;
  int M, N, K;             // END_GATED: N = 2 F, END_GATED_GRAD: N = F
  int F;
  int k_stages;            // K-stages of 64, all of them
  int split_stages;        // ... of one split (blockIdx.y)
  int splits;
  float* part;             // splits > 1: splits x M x part_stride sums (END_GATED: the up projection's in the second half)
  int part_stride;
  int tiles_m, tiles_n;
  const float* factors;    // FACTORS: what column n's sums are multiplied by first (END_GATED: the up projection's from part_stride / 2 on)
};

// Chunk position of 16-byte chunk `c` in a stage row k of an operand that lies
// across k (COLS values a row): pairs of chunks move by an even number that
// differs between the four k-rows one transposing read takes, so that they
// fall on different banks.
template <int COLS>
__device__ __forceinline__ int across_shift(int k) {
  return COLS >= 128 ? 2 * (k & 3) : 2 * ((k >> 1) & 1);
}

// Up to eight consecutive values of a row of `columns`, from column `col` on.
__device__ __forceinline__ void store_columns(uint8_t* C, int out_type, int row, int col, int columns, const float (&v)[8]) {
  const size_t at = (size_t)row * columns + col;
  if (columns % 8 == 0) {
    if (out_type == 0) {
      f32x4* c = (f32x4*)(C + 4 * at);
      c[0] = f32x4{v[0], v[1], v[2], v[3]};
      c[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      *(i32x4*)(C + 2 * at) = out_type == 1 ? narrow8<TypeF16>(v) : narrow8<TypeBF16>(v);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < columns) store_value(C, out_type, at + e, v[e]);
  }
}

// The gradients of eight gates and up values, and h again.
template <typename T>
__device__ __forceinline__ void finish8_grad(const TileArgs& p, int row, int col, const float (&dh)[8], const i32x4& gate, const i32x4& up) {
  const f32x8 g = widen<T>(gate), u = widen<T>(up);
  float dg[8], du[8], h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float act, slope;
    activate_with_slope(g[e], p.activation, act, slope);
    dg[e] = dh[e] * u[e] * slope;
    du[e] = dh[e] * act;
    h[e] = act * u[e];
  }
  uint8_t* const dgu = p.DGU + 2 * ((size_t)row * 2 * p.F + col);
  *(i32x4*)dgu = narrow8<T>(dg);
  *(i32x4*)(dgu + 2 * (size_t)p.F) = narrow8<T>(du);
  *(i32x4*)(p.H + 2 * ((size_t)row * p.F + col)) = narrow8<T>(h);
}

// Eight columns' factors, gate's and up's: loaded ahead of the sums.  (Places up to
// the next multiple of eight columns hold one, too.)
struct Factors8 {
  f32x4 g[2], u[2];
  template <int END>
  __device__ __forceinline__ void load(const TileArgs& p, int col) {
    const float* at = p.factors + col;
    g[0] = *(const f32x4*)at, g[1] = *(const f32x4*)(at + 4);
    if constexpr (END == END_GATED) at += p.part_stride / 2, u[0] = *(const f32x4*)at, u[1] = *(const f32x4*)(at + 4);
  }
  template <int END>
  __device__ __forceinline__ void multiply(float (&v)[8], float (&w)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] *= g[e / 4][e % 4];
      if constexpr (END == END_GATED) w[e] *= u[e / 4][e % 4];
    }
  }
};

// Eight consecutive columns of one row: what END does with them.  `v`: the sums
// (END_GATED: of the gate), `u`: those of the up projection.
template <typename T, int END>
__device__ __forceinline__ void finish8(const TileArgs& p, int row, int col, const float (&v)[8], const float (&u)[8]) {
  if constexpr (END == END_STORE) {
    store_columns(p.C, p.out_type, row, col, p.N, v);
  } else if constexpr (END == END_GATED) {
    float h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = activate(v[e], p.activation) * u[e];
    if (p.GU) {
      uint8_t* gu = p.GU + 2 * ((size_t)row * 2 * p.F + col);
      *(i32x4*)gu = narrow8<T>(v);
      *(i32x4*)(gu + 2 * (size_t)p.F) = narrow8<T>(u);
    }
    store_columns(p.H, p.out_type, row, col, p.F, h);
  } else {
    const uint8_t* gu = p.GU + 2 * ((size_t)row * 2 * p.F + col);
    finish8_grad<T>(p, row, col, v, *(const i32x4*)gu, *(const i32x4*)(gu + 2 * (size_t)p.F));
  }
}

// The splits' sums added in order, eight columns per lane.
template <typename T, int END, bool FACTORS>
__global__ __launch_bounds__(256) void join_splits(TileArgs p) {
  const int columns = END == END_GATED ? p.F : p.N;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int chunks = (columns + 7) / 8;
  const int row = (int)(i / chunks), col = 8 * (int)(i - (int64_t)row * chunks);
  if (row >= p.M) return;
  Factors8 factors;
  if constexpr (FACTORS) factors.template load<END>(p, col);
  float v[8] = {}, u[8] = {};
  for (int s = 0; s < p.splits; ++s) {
    const float* part = p.part + ((size_t)s * p.M + row) * p.part_stride + col;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const f32x4 a = *(const f32x4*)(part + 4 * q);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * q + e] += a[e];
      if constexpr (END == END_GATED) {
        const f32x4 b = *(const f32x4*)(part + p.part_stride / 2 + 4 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e) u[4 * q + e] += b[e];
      }
    }
  }
  if constexpr (FACTORS) factors.template multiply<END>(v, u);
  finish8<T, END>(p, row, col, v, u);
}

template <typename F, int... T>
__device__ __forceinline__ void for_each_slot(F&& f, std::integer_sequence<int, T...>) {
  (f(std::integral_constant<int, T>()), ...);
}

// 16 bytes per lane from buffer offset voff + soff to lds_addr + IMM + 16 lane.
// (M0 is set in one instruction and not restored, the offset along k travels in
// a scalar register: three instructions a load instead of nine, which then fit
// beside the matrix instruction in front of it.)
template <int IMM>
__device__ __forceinline__ void lds_dma_16_at(const i32x4& rsrc, uint32_t lds_addr, uint32_t voff, uint32_t soff) {
  asm volatile(
      "s_add_u32 m0, %0, %4\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds_addr), "v"(voff), "s"(rsrc), "s"(soff), "n"(IMM)
      : "memory", "m0", "scc");
}

// BM x BN tiles, four waves in a WM x WN grid, rings of SA and SB K-stages of 64
// for the two operands.  A stage holds an operand's rows of 128 bytes along k, or its 64 k-rows
// across it; both arrive by 16-byte direct-to-LDS loads, swizzled, and leave
// as 32 x 16 fragments: one ds_read_b128, or two transposing ds_read_b64.  Lane
// l has k = 32 (l / 32) + 8 kk .. + 7 of the stage in K-step kk for both.
//
// One barrier per stage.  The fragments are read three K-steps ahead of their
// products, so that neither their latency nor the wait behind the barrier idles
// the matrix cores; the order of products, reads and loads is pinned (left to the
// compiler the backward pass of 4096 x 4096 x 14336 bf16 takes 2570 us, pinned
// 2480, three K-steps ahead 2445).
//
// Several rounds of 256 x 256 tiles keep the matrix cores busy for 69 to 79% of the
// time (at that size gate and up 69, down 75, dX 79: 689 us, 1396 TFLOP/s), K =
// 4096 rows in the weights' gradients for less (dW_gate_up 66: 775 us, 1241
// TFLOP/s; dW_down 57: 417, 1153): each tile's first loads and its stores are not
// covered by another's products.  The gradients' end reads and writes 587 MB
// between its products (39%; 563 us in all, 372 for the product alone), and 896
// tiles are 3.5 rounds of 256.  A third stage
// for B (160 KB of LDS are used in all) takes 1200 us of both forward products to
// 1171; a third for A does not fit.  Small tiles: 0.43 us a stage of 64 x 128, which
// neither a deeper ring nor earlier fragments shorten.
//
// END_GATED: a wave's columns are WTN / 2 of the gate and the same of the up
// projection, so that both sums of an element meet in one lane.
//
// FACTORS: B's rows were divided by powers of two (4-bit weights); the sums are
// multiplied by them again, which are loaded in front of the main loop (2048 x 64 x
// 256 7.7 -> 7.0 us).  A choice at compile time, in translation units of
// their own: a test of the pointer at run time costs every other product 1 to 5%
// (forward 1024 x 2048 x 5632 86.6 -> 90.8 us), and the same code object its
// neighbours up to 4% (backward of that size 210 -> 218).
template <typename T, bool A_ACROSS, bool B_ACROSS, int BM, int BN, int WM, int WN, int SA, int SB, int END, bool FACTORS>
__global__ __launch_bounds__(256) void ffn_tile(TileArgs p) {
  using Layout = RowLayout<128>;
  constexpr int WTM = BM / WM, WTN = BN / WN;
  constexpr int TM = WTM / 32, TN = WTN / 32;
  static_assert(WM * WN == 4 && TM >= 1 && TN >= 1 && WTM % 32 == 0 && WTN % 32 == 0, "wave tiles");
  static_assert(END != END_GATED || (!B_ACROSS && TN % 2 == 0), "gate and up columns in one wave");
  constexpr bool GATED = END == END_GATED;
  constexpr int kStageA = BM * 128, kStageB = BN * 128, kRingB = SA * kStageA;
  constexpr int kSlots = (BM + BN) / 32, kSlotsA = BM / 32, kSlotsB = BN / 32;   // 1 KiB loads per wave and stage
  constexpr int kLds = kRingB + SB * kStageB;
  static_assert(kLds <= 160 * 1024, "LDS");
  // loads that may be in flight once stage s + 1 has landed: those behind the
  // later of A's and B's, which go out in rounds s + 1 - SA and s + 1 - SB, A's
  // before B's
  static_assert(SB >= SA && SA >= 2, "rings");
  constexpr int kInFlight = (SA - 2) * kSlots + (SB > SA ? kSlotsB : 0);
  static_assert(kInFlight + kSlots <= 63, "vmcnt range");

  __shared__ __attribute__((aligned(1024))) uint8_t smem[kLds];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  // bands of 8 row tiles, column tile by column tile; every XCD a contiguous range
  const int logical = xcd_logical(blockIdx.x, p.tiles_m * p.tiles_n);
  const int band = logical / (8 * p.tiles_n), in_band = logical - band * 8 * p.tiles_n;
  const int height = min(p.tiles_m - 8 * band, 8);
  const int m0 = (8 * band + in_band % height) * BM;
  constexpr int kTileColumns = GATED ? BN / 2 : BN;
  const int n0 = (in_band / height) * kTileColumns;
  const int columns = GATED ? p.F : p.N;
  const int rows = min(BM, p.M - m0), cols = min(kTileColumns, columns - n0);

  const int s_begin = blockIdx.y * p.split_stages;
  const int s_end = min(s_begin + p.split_stages, p.k_stages);

  const uint8_t* const a_base = A_ACROSS ? p.A + 2 * (size_t)m0 : p.A + (size_t)m0 * p.a_stride;
  const uint8_t* const b_base = B_ACROSS ? p.B + 2 * (size_t)n0 : p.B + (size_t)n0 * p.b_stride;
  const uint32_t smem_lds = lds_address(smem);

  // Load slot t of this wave fills 1 KiB of a stage.  Along k: stage rows 32 t +
  // 8 wave .. + 7, eight lanes a row.  Across: 1024 / (2 BX) k-rows.  A lane
  // fetches the chunk whose swizzled place is its own.
  const int lrow = 8 * wave + lane / 8;
  const uint32_t along_col = Layout::pos(lrow, lane % 8) * 16;   // (rows 32 apart have the same swizzle)
  uint32_t off[kSlots];
#pragma unroll
  for (int t = 0; t < kSlots; ++t) {
    const bool is_a = t < kSlotsA;
    const int u = is_a ? t : t - kSlotsA;
    if (is_a ? A_ACROSS : B_ACROSS) {
      const int bx = is_a ? BM : BN, per_row = bx / 8;
      const int k = (4 * u + wave) * (64 / per_row) + lane / per_row, at = lane % per_row;
      const int shift = is_a ? across_shift<BM>(k) : across_shift<BN>(k);
      const int c = (((at >> 1) ^ shift) << 1) | (at & 1);
      off[t] = 8 * c < (is_a ? rows : cols) ? (uint32_t)(k * (is_a ? p.a_stride : p.b_stride)) + 16 * c : kOutOfRange;
    } else if (is_a || !GATED) {
      off[t] = (uint32_t)((32 * u + lrow) * (is_a ? p.a_stride : p.b_stride)) + along_col;
    } else {   // 32-row block u of B: gate or up columns of wave column 32 u / WTN
      const int c = 32 * u / WTN * (WTN / 2) + 32 * u % (WTN / 2) + lrow;
      off[t] = (uint32_t)(c * p.b_stride) + along_col;
    }
  }
  const bool has_up = GATED;
  const uint32_t row_bytes = 2 * (uint32_t)p.K;
  const i32x4 rsrc_a_along = make_rsrc(a_base, A_ACROSS ? 0 : (uint32_t)(rows * p.a_stride));
  const i32x4 rsrc_b_along = make_rsrc(b_base, B_ACROSS ? 0 : (uint32_t)(cols * p.b_stride));
  const i32x4 rsrc_up = make_rsrc(has_up ? b_base + (size_t)p.F * p.b_stride : b_base, has_up ? (uint32_t)(cols * p.b_stride) : 0);
  // across k, a stage's k-rows have a descriptor of their own: the whole operand may be larger than 4 GiB
  auto across_rsrc = [&](const uint8_t* base, int64_t stride, int s) {
    const int left = s < s_end ? min(p.K - 64 * s, 64) : 0;
    return make_rsrc(base + (int64_t)64 * s * stride, (uint32_t)(left * stride));
  };
  i32x4 rsrc_a = rsrc_a_along, rsrc_b = rsrc_b_along;
  auto enter_stage = [&](int sa, int sb) {   // the descriptors for the loads of these stages
    if constexpr (A_ACROSS) rsrc_a = across_rsrc(a_base, p.a_stride, sa);
    if constexpr (B_ACROSS) rsrc_b = across_rsrc(b_base, p.b_stride, sb);
  };
  // Along k: a scalar offset, no records past the last stage, and lanes whose
  // chunk lies behind the row's end in the stage where it ends.  t: the load slot.
  const uint32_t wave_lds = smem_lds + wave * 1024;
  auto issue_load = [&](auto t_c, int s, int slot) __attribute__((always_inline)) {   // of stage s, into that place of the ring
    constexpr int t = decltype(t_c)::value;
    constexpr bool is_a = t < kSlotsA;
    constexpr int u = is_a ? t : t - kSlotsA;
    const uint32_t ring = wave_lds + (is_a ? slot * kStageA : kRingB + slot * kStageB);
    if constexpr (is_a ? A_ACROSS : B_ACROSS) {
      lds_dma_16_at<4096 * u>(is_a ? rsrc_a : rsrc_b, ring, off[t], 0);
    } else {
      // (past the last stage: no records, and a scalar offset of 0, as the range
      // check may take it off the records)
      const uint32_t kbyte = s < s_end ? (uint32_t)s * 128 : 0;
      const uint32_t from = along_col < row_bytes - kbyte ? off[t] : kOutOfRange;
      constexpr bool up = !is_a && GATED && (32 * u) % WTN >= WTN / 2;
      i32x4 rsrc = is_a ? rsrc_a : up ? rsrc_up : rsrc_b;
      if (s >= s_end) rsrc.z = 0;
      lds_dma_16_at<4096 * u>(rsrc, ring, from, kbyte);
    }
  };

  // fragment addresses of this lane within a stage, in K-step 0
  const int fr = lane & 31, fh = lane >> 5;
  uint32_t a_at[A_ACROSS ? TM : 1], b_at[B_ACROSS ? TN : 1];
  auto across_at = [&](int bx, int block, int shift) {   // block: of 32 columns
    const int i = lane & 15, k = 32 * fh + (i >> 2);
    return (uint32_t)(k * 2 * bx + (((2 * block) ^ shift) + ((lane >> 4) & 1)) * 32 + 8 * (i & 3));
  };
  if constexpr (A_ACROSS) {
#pragma unroll
    for (int i = 0; i < TM; ++i) a_at[i] = smem_lds + across_at(BM, wm * TM + i, across_shift<BM>((lane & 15) >> 2));
  } else {
    a_at[0] = 0;
  }
  if constexpr (B_ACROSS) {
#pragma unroll
    for (int j = 0; j < TN; ++j) b_at[j] = smem_lds + kRingB + across_at(BN, wn * TN + j, across_shift<BN>((lane & 15) >> 2));
  } else {
    b_at[0] = 0;
  }

  i32x4 fa[4][TM], fb[4][TN];   // of four K-steps
  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  auto read_across = [&](uint32_t at, int bx) {
    const u32x2 lo = lds_read_transposed16(at), hi = lds_read_transposed16(at + 8 * bx);
    return i32x4{(int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y};
  };
  // fragment n of K-step kk, in the order the products need them: A's first, B's, A's others
  constexpr int kFrags = TM + TN;
  auto read_frag = [&](int n, int slot_a, int slot_b, int kk) __attribute__((always_inline)) {
    const uint8_t* base = smem + Layout::off(fr, 4 * fh + kk);
    if (n >= 1 && n <= TN) {
      const int j = n - 1;
      if constexpr (B_ACROSS) fb[kk][j] = read_across(b_at[j] + slot_b * kStageB + kk * 16 * BN, BN);
      else fb[kk][j] = *(const i32x4*)(base + kRingB + slot_b * kStageB + (wn * TN + j) * 4096);
    } else {
      const int i = n == 0 ? 0 : n - TN;
      if constexpr (A_ACROSS) fa[kk][i] = read_across(a_at[i] + slot_a * kStageA + kk * 16 * BM, BM);
      else fa[kk][i] = *(const i32x4*)(base + slot_a * kStageA + (wm * TM + i) * 4096);
    }
  };
  constexpr int kMfma = TM * TN;
  auto product = [&](int x, int kk) __attribute__((always_inline)) {
    acc[x / TN][x % TN] = mfma32<T>(fb[kk][x % TN], fa[kk][x / TN], acc[x / TN][x % TN]);
  };
  auto each_slot = [](auto&& f) __attribute__((always_inline)) { for_each_slot(f, std::make_integer_sequence<int, kSlots>()); };
  // A round: stage s + 1 has landed and everyone has read stage s, whose places
  // then take stages s + SA and s + SB; K-steps 1, 2, 3 of stage s and 0 of stage
  // s + 1 run, and the fragments of stage s + 1 are read, three K-steps ahead.
  constexpr int kReadSpan = kMfma > 8 ? kFrags : kMfma;
  int slot_a = 0, slot_b = 0;   // the places of stage s
  auto round = [&](int s, auto first_c) __attribute__((always_inline)) {
    constexpr bool first = decltype(first_c)::value;   // in front of the first stage: no products yet
    wait_vmcnt<kInFlight>();   // own loads of stage s + 1 landed
    wait_lgkmcnt0();           // own reads of stage s done
    block_barrier();           // ... everyone's
    const int next_a = slot_a == SA - 1 ? 0 : slot_a + 1, next_b = slot_b == SB - 1 ? 0 : slot_b + 1;
    enter_stage(s + SA, s + SB);   // (past the last stage the loads move no data)
    auto step = [&](auto j_c) __attribute__((always_inline)) {
      constexpr int j = decltype(j_c)::value, kk = (j + 1) % 4;
      // product x, then what goes out behind it
      auto one = [&](auto x_c) __attribute__((always_inline)) {
        constexpr int x = decltype(x_c)::value;
        if constexpr (!first || j == 3) product(x, kk);
        if constexpr (x < kReadSpan) {
#pragma unroll
          for (int n = x * kFrags / kReadSpan; n < (x + 1) * kFrags / kReadSpan; ++n) read_frag(n, next_a, next_b, j);
        }
        each_slot([&](auto t_c) __attribute__((always_inline)) {
          constexpr int t = decltype(t_c)::value;
          // A's in the first K-step, B's in the next two
          constexpr int per = t < kSlotsA ? kSlotsA : (kSlotsB + 1) / 2, at = t < kSlotsA ? 0 : 1 + (t - kSlotsA) / per, l = t < kSlotsA ? t : (t - kSlotsA) % per;
          if constexpr (at == j && (2 * l + 1) * kMfma / (2 * per) == x)
            issue_load(t_c, t < kSlotsA ? s + SA : s + SB, t < kSlotsA ? slot_a : slot_b);
        });
        __builtin_amdgcn_sched_barrier(0);
      };
      for_each_slot(one, std::make_integer_sequence<int, kMfma>());
    };
    step(std::integral_constant<int, 0>());
    step(std::integral_constant<int, 1>());
    step(std::integral_constant<int, 2>());
    step(std::integral_constant<int, 3>());
    slot_a = next_a;
    slot_b = next_b;
  };

  constexpr int kBlocks = GATED ? TN / 2 : TN;   // column blocks of C
  const int wave_col = n0 + wn * (GATED ? WTN / 2 : WTN) + 8 * fh;
  Factors8 factors[FACTORS ? 2 * kBlocks : 1];   // (the loads land behind the main loop)
  if constexpr (FACTORS) {
#pragma unroll
    for (int c = 0; c < 2 * kBlocks; ++c) factors[c].template load<END>(p, wave_col + 16 * c < columns ? wave_col + 16 * c : 0);
  }

  if (s_begin < s_end) {
    // the loads that the rounds before would have sent
#pragma unroll
    for (int i = -SB; i < -1; ++i) {
      enter_stage(s_begin + i + SA, s_begin + i + SB);
      each_slot([&](auto t_c) __attribute__((always_inline)) {
        if (decltype(t_c)::value >= kSlotsA) issue_load(t_c, s_begin + i + SB, i + SB);
        else if (i + SA >= 0) issue_load(t_c, s_begin + i + SA, i + SA);
      });
    }
    slot_a = SA - 1;
    slot_b = SB - 1;
    round(s_begin - 1, std::true_type());
    // (the last round's last K-step is of a stage of zeros)
    for (int s = s_begin; s < s_end; ++s) round(s, std::false_type());
  }

  wait_vmcnt<0>();   // (loads past the last stage: LDS is the next workgroup's once this one ends)
  // The matrix instructions have B's rows as theirs: a lane holds one row of C,
  // and of its columns four at a time, 8 q + 4 (l / 32) .. + 3 of each 32.  Two
  // such runs, exchanged between the half-waves, are eight consecutive columns.
  auto eight = [&](const f32x16& x, int q, float (&v)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lo = x[8 * q + e], hi = x[8 * q + 4 + e];
      const u32x2 t = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi), false, false));
      const uint32_t first = t.x, second = t.y;
      v[e] = __builtin_bit_cast(float, first);
      v[4 + e] = __builtin_bit_cast(float, second);
    }
  };
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int row = m0 + wm * WTM + 32 * i + fr;
    __builtin_amdgcn_sched_barrier(0);   // (else the compiler reads every accumulator out at once)
#pragma unroll
    for (int j = 0; j < TN; ++j) asm volatile("" : "+a"(acc[i][j]));
    i32x4 kept[END == END_GATED_GRAD ? 4 * kBlocks : 1];   // g and u of the block's chunks, loaded together
    if constexpr (END == END_GATED_GRAD) {
#pragma unroll
      for (int c = 0; c < 2 * kBlocks; ++c) {
        const int col = wave_col + 16 * c;
        if (p.splits == 1 && row < p.M && col < columns) {
          const uint8_t* gu = p.GU + 2 * ((size_t)row * 2 * p.F + col);
          kept[2 * c] = *(const i32x4*)gu;
          kept[2 * c + 1] = *(const i32x4*)(gu + 2 * (size_t)p.F);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < 2 * kBlocks; ++c) {
      const int col = wave_col + 16 * c;
      float v[8], u[8] = {};
      eight(acc[i][c / 2], c % 2, v);
      if constexpr (GATED) eight(acc[i][c / 2 + kBlocks], c % 2, u);
      if (row >= p.M || col >= columns) continue;
      if (p.splits > 1) {
        f32x4* part = (f32x4*)(p.part + ((size_t)blockIdx.y * p.M + row) * p.part_stride + col);
        part[0] = f32x4{v[0], v[1], v[2], v[3]};
        part[1] = f32x4{v[4], v[5], v[6], v[7]};
        if constexpr (GATED) {
          part = (f32x4*)((float*)part + p.part_stride / 2);
          part[0] = f32x4{u[0], u[1], u[2], u[3]};
          part[1] = f32x4{u[4], u[5], u[6], u[7]};
        }
      } else if constexpr (END == END_GATED_GRAD) {
        finish8_grad<T>(p, row, col, v, kept[2 * c], kept[2 * c + 1]);
      } else {
        if constexpr (FACTORS) factors[c].template multiply<END>(v, u);
        finish8<T, END>(p, row, col, v, u);
      }
    }
  }
}

}  // namespace lpgemm
