// Products grouped by expert, and the MXFP4 product (one group).
//
//   C[i] = A[row_index[i]] . B_g     for the rows i of group g
//
// Two kernel families, both with K-contiguous operand rows moved by 16-byte
// direct-to-LDS loads into XOR-swizzled 128-byte LDS rows (RowLayout<128>)
// and 32 x 32 MFMAs (16 operand bytes per lane and step: 32 int8, 16
// binary16 or 64 E2M1 values of k):
//
//   grouped_tile    BM x BN tiles, four waves, a ring of K-stages
//   grouped_skinny  32 columns per workgroup, whose waves split K: for few
//                   rows per group, where the weights' stream is the work
//
// A workgroup finds its tile on the device: a grid for the largest number of
// tiles the sizes allow is launched, every wave scans the groups' offsets
// for the row tiles each group has, and workgroups past the last tile leave.
#pragma once

#include "gemm_kernels.hpp"

namespace lpgemm {

constexpr int KIND_MXFP4 = 6;   // beside enum Kind: E2M1 codes with E8M0 scales

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x8_t __attribute__((ext_vector_type(8)));

struct GroupedArgs {
  const uint8_t* A;          // rows of row_bytes
  const uint8_t* B;          // groups x N rows of row_bytes
  const uint8_t* a_scale;    // MXFP4: rows of scale_stride bytes
  const uint8_t* b_scale;
  const float* row_scale;    // int8: one per row of A
  const float* col_scale;    // int8: groups x N
  const int32_t* offsets;    // groups + 1 (null: one group of all rows)
  const int32_t* row_index;  // rows (null: row i is A's row i)
  uint8_t* C;
  int out_type;              // lpgemm_type of C
  int rows, a_rows, groups, N;
  int row_bytes;
  int scale_stride;
  int k_stages;              // 128-byte K-stages
  int tiles_n;
  int tile_w;                // grouped_skinny: columns per workgroup, at most 32
};

// This workgroup's tile: rows [row0, row_end) of C (at most the tile's), all
// of group `group`, and column tile tn.
struct GroupTile {
  int group, row0, row_end, tn;
  bool none;
};

// Tile `in_group` of a group of rows [first, end) in tm_count row tiles: bands
// of 8 row tiles, column tile by column tile.
template <int BM>
__device__ __forceinline__ void place_tile(const GroupedArgs& p, int in_group, int tm_count, int first, int end,
                                           GroupTile& t) {
  if (in_group < 0) return;
  const int band = in_group / (8 * p.tiles_n);
  const int in_band = in_group - band * 8 * p.tiles_n;
  const int height = min(tm_count - 8 * band, 8);
  if (height <= 0) return;
  const int tm = 8 * band + in_band % height;
  if (tm < 0 || tm >= tm_count) return;
  t.tn = in_band / height;
  t.row0 = first + tm * BM;
  t.row_end = min(end, t.row0 + BM);
  t.none = false;
}

// Row tiles of group g, and its first row and end, with the offsets clamped
// to the rows there are.
template <int BM>
__device__ __forceinline__ int group_tiles(const GroupedArgs& p, int g, int& first, int& end) {
  first = end = 0;
  if (g >= p.groups) return 0;
  first = min(max(p.offsets[g], 0), p.rows);
  end = min(max(p.offsets[g + 1], 0), p.rows);
  return end > first ? (end - first + BM - 1) / BM : 0;
}

__device__ __forceinline__ int wave_inclusive_sum(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int x = __shfl_up(v, off);
    if (lane >= off) v += x;
  }
  return v;
}

// The tiles in order: group by group; within a group bands of 8 row tiles,
// column tile by column tile (so that workgroups running together share the
// group's weights and a few rows' operands in an XCD's L2; every XCD takes a
// contiguous range).  64 groups are scanned at a time, one per lane.
template <int BM>
__device__ __forceinline__ GroupTile find_tile(const GroupedArgs& p, int w) {
  const int lane = threadIdx.x & 63;
  GroupTile t;
  t.none = true;
  t.group = t.row0 = t.row_end = t.tn = 0;
  if (!p.offsets) {   // one group of all rows
    const int count = (p.rows + BM - 1) / BM;
    if (w >= count * p.tiles_n) return t;
    place_tile<BM>(p, xcd_logical(w, count * p.tiles_n), count, 0, p.rows, t);
    return t;
  }
  int first = 0, end = 0;
  int mine = group_tiles<BM>(p, lane, first, end);
  int upto = wave_inclusive_sum(mine);
  int total = __builtin_amdgcn_readlane(upto, 63);
  for (int g0 = 64; g0 < p.groups; g0 += 64) {
    int f, e;
    total += __builtin_amdgcn_readlane(wave_inclusive_sum(group_tiles<BM>(p, g0 + lane, f, e)), 63);
  }
  const int nb = total * p.tiles_n;
  if (w >= nb) return t;
  const int logical = xcd_logical(w, nb);
  const int unit = logical / p.tiles_n;   // counts row tiles: a group's tiles are consecutive
  int before = 0;
  for (int g0 = 0; g0 < p.groups; g0 += 64) {
    if (g0 > 0) {
      mine = group_tiles<BM>(p, g0 + lane, first, end);
      upto = wave_inclusive_sum(mine);
    }
    const uint64_t past = __ballot(before + upto > unit);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      const int tm_count = __builtin_amdgcn_readlane(mine, l);
      const int tiles_before = before + __builtin_amdgcn_readlane(upto, l) - tm_count;
      const int gfirst = __builtin_amdgcn_readlane(first, l);
      const int gend = __builtin_amdgcn_readlane(end, l);
      // (counts of overlapping groups may wrap: place_tile checks)
      place_tile<BM>(p, logical - tiles_before * p.tiles_n, tm_count, gfirst, gend, t);
      t.group = g0 + l;
      return t;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return t;
}

// Operand row of A behind row i of C: -1 where there is none.
__device__ __forceinline__ int a_row_of(const GroupedArgs& p, int i, int row_end) {
  if (i >= row_end) return -1;
  if (!p.row_index) return i;
  const int r = p.row_index[i];
  return (uint32_t)r < (uint32_t)p.a_rows ? r : -1;
}

template <int KIND>
struct GroupedAcc {
  using type = f32x16;
};
template <>
struct GroupedAcc<KIND_I8_DEQUANT> {
  using type = i32x16;
};

// One 32 x 32 MFMA step on 16 operand bytes per lane; MXFP4: 64 values of k,
// this lane's block scale in byte STEP of its scale word.
template <int KIND, int STEP>
__device__ __forceinline__ typename GroupedAcc<KIND>::type grouped_mfma(const i32x4& a, const i32x4& b,
                                                                       const typename GroupedAcc<KIND>::type& c,
                                                                       int sa, int sb) {
  if constexpr (KIND == KIND_MXFP4) {
    const i32x8 a8 = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8 b8 = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, STEP, sa, STEP, sb);
  } else if constexpr (KIND == KIND_F16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  } else {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
  }
}

// The scale bytes of blocks 4 h .. 4 h + 3 of K-stage s (eight blocks of 32
// values) that lie inside the row; the others, padding, become 2^-127 (their
// codes are zero, but a padding byte of 255 would be a NaN).
__device__ __forceinline__ int scale_mask(int s, int h, int blocks) {
  const int left = blocks - 8 * s - 4 * h;
  return left >= 4 ? -1 : (left <= 0 ? 0 : (int)((1u << (8 * left)) - 1));
}

// Consecutive columns' binary32 results as 16 bytes of C: 4 in binary32, 8 in
// a 16-bit type.  The kernel does not read C again: the stores are
// non-temporal (MXFP4 2048 x 4096 x 4096 23.8 against 25.5 us, with the
// activation that reads C behind it 29.1 against 30.4; int8 8192 x 14336 x
// 4096 421 against 435, 477 against 486).
template <int COLS>
__device__ __forceinline__ void store16(const GroupedArgs& p, size_t idx, const float (&v)[COLS]) {
  if constexpr (COLS == 4) {
    __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, (f32x4_t*)(p.C + 4 * idx));
  } else {
    const f32x8_t w = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
    const i32x4 h = p.out_type == 1 ? __builtin_bit_cast(i32x4, __builtin_convertvector(w, f16x8))
                                    : __builtin_bit_cast(i32x4, __builtin_convertvector(w, bf16x8_t));
    __builtin_nontemporal_store(h, (i32x4*)(p.C + 2 * idx));
  }
}
__device__ __forceinline__ void store1(const GroupedArgs& p, size_t idx, float v) {
  if (p.out_type == 0) ((float*)p.C)[idx] = v;
  else if (p.out_type == 1) ((_Float16*)p.C)[idx] = (_Float16)v;
  else ((__bf16*)p.C)[idx] = (__bf16)v;
}

// ---------------------------------------------------------------------------
// BM x BN tiles, 4 waves in a WM x WN grid, STAGES K-stages of 128 bytes per
// operand row.  The loads of stage s + STAGES - 1 go out during stage s; one
// barrier per stage, in the middle of its last K-step, publishes stage s + 1,
// whose first fragments are read while the rest of stage s's MFMAs run.
//
// Lane l of a fragment reads row l % 32, chunk 4 (l / 32) + kk of the stage
// row in K-step kk, for A and B alike, so the half-wave of a lane sees four
// consecutive MXFP4 blocks per stage: one 32-bit word of scale bytes, of
// which step kk uses byte kk.
//
// MXFP4 scales travel with the operands: every fourth stage two 16-byte loads
// per operand row fetch the scales of four stages (32 blocks, 32 bytes) into
// one of two buffers of their own (a row's scales lie in one cache line per
// 4096 values of k, which every fetch moves again: with 16 bytes per fetch
// 8192^3 took 307 us, without any scale loads 273), two stages ahead; they are
// read a stage ahead, in a K-step that waits for nothing else (read behind the
// stage barrier: 267 us against 260).
//
// The loads of a stage all go out in its first two K-steps (MXFP4 2048 x 4096
// x 4096 on 128 x 128 tiles 22.4 us, over three 23.3; 8192^3 on 256 x 256 in
// one 264, in two 250).  PIN: one MFMA is pinned in front of each (the schedule
// would otherwise issue them back to back: 8192^3 272 us against 265).
//
// TAIL: a group's last tile runs the main loop for the 32-row blocks that its
// rows reach, in steps of WM blocks; its loads and products for the other
// rows are left out.  There the waves' rows alternate by block, so that the
// blocks fall on all of them; in a whole tile each wave has one run of rows
// (alternating there too took 8192^3 from 272 to 279 us).  Needs two stages.
//
// BNT: B streams non-temporally, where it is read once.
//
// Bound by operand latency and power where a tile has many rows (256 x 256:
// MXFP4 8192^3 259 us, 4.2 PFLOP/s, without its operand loads 210; int8, 8
// experts of 1024 rows, 14336 x 4096, 524 to 541 us on several cards, 1.8
// POP/s), by the weights where it has few (MXFP4, 64 experts of 32 rows, 2048 x
// 4096, 54 to 63 us, 4.7 to 5.5 TB/s), and in between, where a CU gets one or
// two tiles of 100 rows and more, by the latency of each stage, which two
// stages do not hide (int8, 4 experts of 242 rows each, 4096 x 4096, 37.5 us,
// of 120 to 300 rows 44.9, 1.2 and 1.4 a stage; the floor is 15.6).
template <int KIND, int BM, int BN, int WM, int WN, int STAGES, bool PIN, bool TAIL, bool BNT = false>
__global__ __launch_bounds__(256) void grouped_tile(GroupedArgs p) {
  using Acc = typename GroupedAcc<KIND>::type;
  using Layout = RowLayout<128>;
  constexpr bool MX = KIND == KIND_MXFP4;
  constexpr int WTM = BM / WM, WTN = BN / WN;
  constexpr int TM = WTM / 32, TN = WTN / 32;
  static_assert(WM * WN == 4 && TM >= 1 && TN >= 1 && WTM % 32 == 0 && WTN % 32 == 0, "wave tiles");
  constexpr int kRows = BM + BN;
  constexpr int kStage = kRows * 128;
  static_assert(kRows % 32 == 0 && BM % 32 == 0, "loads per wave");
  constexpr int kSlots = kRows / 32;          // 1 KiB loads per wave per stage (8 rows each)
  constexpr int kSlotsA = BM / 32;
  constexpr int kSc = MX ? (kRows / 32 + 3) / 4 : 0;   // scale loads per wave, every fourth stage (32 rows each)
  constexpr int kScBuf = kSc * 4096;
  // Two buffers.  The scales of stages 4 e + 4 .. 4 e + 7 are fetched at the
  // start of stage 4 e + 1, into the buffer last read during stage 4 e - 2.
  // They are read from stage 4 e + 3 on, and have landed by the end of stage
  // 4 e + 2: at most the loads of the STAGES - 2 stages issued behind them
  // may then be in flight.
  static_assert(!MX || (STAGES >= 2 && STAGES <= 4), "scale buffers");
  static_assert(!TAIL || STAGES == 2, "fewer loads in flight than the waits of a longer ring count");
  constexpr int kMainLds = STAGES * kStage + 2 * kScBuf;
  constexpr int kEpiPitch = WTN * 4 + 32;
  constexpr int kEpiRows = WTM < 64 ? WTM : 64;
  constexpr int kEpiWave = kEpiRows * kEpiPitch;
  constexpr int kLds = kMainLds > 4 * kEpiWave ? kMainLds : 4 * kEpiWave;
  static_assert(kLds <= 160 * 1024, "LDS");
  // loads that may be in flight once stage s + 1 has landed: those of stages
  // s + 2 .. s + STAGES - 1
  constexpr int kInFlight = (STAGES - 2) * kSlots;
  static_assert(kInFlight + kSlots + kSc <= 63, "vmcnt range");

  __shared__ __attribute__((aligned(1024))) uint8_t smem[kLds];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;

  const GroupTile tile = find_tile<BM>(p, blockIdx.x);
  if (tile.none) return;
  const int n0 = tile.tn * BN;
  const int cols = min(BN, p.N - n0);
  const size_t brow0 = (size_t)tile.group * p.N + n0;   // first row of B
  // gathered rows: the whole of A (below 2 GiB), else this tile's rows
  const bool gather = p.row_index != nullptr;
  const size_t arow0 = gather ? 0 : tile.row0;
  const int arows = gather ? p.a_rows : tile.row_end - tile.row0;
  const i32x4 rsrc_a = make_rsrc(p.A + arow0 * p.row_bytes, (uint32_t)arows * p.row_bytes);
  const i32x4 rsrc_b = make_rsrc(p.B + brow0 * p.row_bytes, (uint32_t)cols * p.row_bytes);
  const i32x4 rsrc_as = make_rsrc(MX ? p.a_scale + arow0 * p.scale_stride : p.A, MX ? (uint32_t)arows * p.scale_stride : 0);
  const i32x4 rsrc_bs = make_rsrc(MX ? p.b_scale + brow0 * p.scale_stride : p.B, MX ? (uint32_t)cols * p.scale_stride : 0);
  const uint32_t smem_lds = lds_address(smem);

  // operand row of the tile's row r (A's rows first): a row of the buffer
  // above, or -1
  auto source_row = [&](int r) -> int {
    if (r >= BM) return r - BM;
    return gather ? a_row_of(p, tile.row0 + r, tile.row_end) : r;
  };
  // Load slot t of this wave fills stage rows 8 g .. 8 g + 7, g = 4 t + wave:
  // lane l writes row 8 g + l / 8 at chunk position l % 8, so it fetches the
  // chunk whose swizzled position that is.
  uint32_t slot_off[kSlots];
  uint32_t slot_col;
  {
    const int lrow0 = 8 * wave + lane / 8;   // rows 32 apart have the same swizzle
    slot_col = Layout::pos(lrow0, lane % 8) * 16;
#pragma unroll
    for (int t = 0; t < kSlots; ++t) {
      const int r = source_row(32 * t + lrow0);
      slot_off[t] = r < 0 ? kOutOfRange : (uint32_t)r * (uint32_t)p.row_bytes + slot_col;
    }
  }
  // scale slot t of this wave: rows 32 (4 t + wave) + lane / 2, 16 of their 32
  // bytes; the halves of every second 8 rows change places, so that the words
  // of 16 consecutive rows lie in different banks (those of rows 16 apart do
  // not)
  const int sc_half = ((lane & 1) ^ ((lane >> 4) & 1)) * 16;
  uint32_t sc_off[MX ? kSc : 1];
  if constexpr (MX) {
#pragma unroll
    for (int t = 0; t < kSc; ++t) {
      const int r = 32 * (4 * t + wave) + lane / 2;
      const int src = r < kRows ? source_row(r) : -1;
      sc_off[t] = src < 0 ? kOutOfRange : (uint32_t)src * (uint32_t)p.scale_stride + sc_half;
    }
  }
  auto issue_load = [&](int t, int s) {
    const uint32_t kbyte = (uint32_t)s * 128;
    const uint32_t off = kbyte + slot_col < (uint32_t)p.row_bytes ? slot_off[t] + kbyte : kOutOfRange;
    const uint32_t to = smem_lds + (s % STAGES) * kStage + (4 * t + wave) * 1024;
    if (t < kSlotsA) lds_dma_16(rsrc_a, to, off);
    else lds_dma_16<BNT ? 1 : 0>(rsrc_b, to, off);
  };
  auto issue_scales = [&](int e) {   // of stages 4 e .. 4 e + 3: blocks 32 e .. 32 e + 31 of every row
    if constexpr (MX) {
      const bool inside = 32 * e + sc_half < p.scale_stride;
#pragma unroll
      for (int t = 0; t < kSc; ++t) {
        const uint32_t off = inside ? sc_off[t] + 32 * e : kOutOfRange;
        const uint32_t to = smem_lds + STAGES * kStage + (e & 1) * kScBuf + (4 * t + wave) * 1024;
        if (32 * (4 * t + wave) < BM) lds_dma_16(rsrc_as, to, off);
        else lds_dma_16(rsrc_bs, to, off);
      }
    }
  };

  const int fr = lane & 31, fh = lane >> 5;
  // block i of a wave is the tile's 32-row block step i + base: the wave's own
  // run of rows, or, in a partial tile, every WM-th block
  const int used_blocks = TAIL ? (tile.row_end - tile.row0 + 32 * WM - 1) / (32 * WM) : TM;
  const bool partial = TAIL && used_blocks < TM;
  const int b_base = (BM + wn * WTN) * 128;
  i32x4 fa[2][TM], fb[2][TN];
  const int blocks = p.row_bytes / 16;   // MXFP4 blocks of 32 values (16 bytes)
  int sa[TM] = {}, sb[TN] = {}, sa_next[TM] = {}, sb_next[TN] = {};
  Acc acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  constexpr int kLoadSteps = 2;
  constexpr int kLoadsPerStep = (kSlots + kLoadSteps - 1) / kLoadSteps;
  const int nks = p.k_stages;   // 0 when K = 0: C is written as zeros

  // the main loop over the first TMU blocks of every wave
  auto main_loop = [&](auto tmu_c) __attribute__((always_inline)) {
    constexpr int TMU = decltype(tmu_c)::value;
    constexpr int kMfma = TMU * TN;
    constexpr int kStep = TMU == TM ? 1 : WM;
    const int row_base = TMU == TM ? wm * TM : wm;
    const int a_base = row_base * 4096;
    constexpr int kSplit = kMfma > 1 ? kMfma / 2 : 1;
    constexpr int kReads = TMU + TN;
    constexpr int kSlotsUsed = kSlotsA * TMU / TM;   // of A's load slots
    auto used = [](int t) { return t < kSlotsUsed || t >= kSlotsA; };
    auto read_frags = [&](int s, int kk, int dst) {
      const uint8_t* base = smem + (s % STAGES) * kStage + Layout::off(fr, 4 * fh + kk);
#pragma unroll
      for (int i = 0; i < TMU; ++i) fa[dst][i] = *(const i32x4*)(base + a_base + kStep * i * 4096);
#pragma unroll
      for (int j = 0; j < TN; ++j) fb[dst][j] = *(const i32x4*)(base + b_base + j * 4096);
    };
    auto read_scales = [&](int s) {   // of stage s, into sa_next / sb_next
      if constexpr (MX) {
        const uint8_t* base = smem + STAGES * kStage + ((s / 4) & 1) * kScBuf + fr * 32 +
                              ((((s >> 1) ^ (fr >> 3)) & 1) << 4) + (s & 1) * 8 + fh * 4;
#pragma unroll
        for (int i = 0; i < TMU; ++i) sa_next[i] = *(const int*)(base + (kStep * i + row_base) * 1024);
#pragma unroll
        for (int j = 0; j < TN; ++j) sb_next[j] = *(const int*)(base + (BM + wn * WTN + j * 32) * 32);
      }
    };
    auto compute = [&](auto kk_c, int src, int first, int last) {
      constexpr int kk = decltype(kk_c)::value;
#pragma unroll
      for (int x = 0; x < kMfma; ++x) {
        if (x < first || x >= last) continue;
        const int i = x / TN, j = x % TN;
        acc[i][j] = grouped_mfma<KIND, kk>(fa[src][i], fb[src][j], acc[i][j], sa[i], sb[j]);
      }
    };
    auto interleave = [&](int mfmas, int reads, int loads) {
#pragma unroll
      for (int x = 0; x < kMfma; ++x) {
        if (x >= mfmas) break;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                  // MFMA
        if (x < reads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // DS read
        if (x < loads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);   // VMEM read
      }
    };
    if (nks > 0) {
      issue_scales(0);
#pragma unroll
      for (int s = 0; s < STAGES - 1; ++s)
#pragma unroll
        for (int t = 0; t < kSlots; ++t)
          if (used(t)) issue_load(t, s);
      wait_vmcnt<kInFlight>();
      block_barrier();
      read_frags(0, 0, 0);
      read_scales(0);
    }
    for (int s = 0; s < nks; ++s) {
      // loads for stage s + STAGES - 1 (past the last stage they move no data)
      const int sl = s + STAGES - 1;
      if constexpr (MX) {
#pragma unroll
        for (int i = 0; i < TMU; ++i) sa[i] = sa_next[i];
#pragma unroll
        for (int j = 0; j < TN; ++j) sb[j] = sb_next[j];
        if (8 * s + 8 > blocks) {   // the row ends inside the stage: padding bytes follow
          const int mask = scale_mask(s, fh, blocks);
#pragma unroll
          for (int i = 0; i < TMU; ++i) sa[i] &= mask;
#pragma unroll
          for (int j = 0; j < TN; ++j) sb[j] &= mask;
        }
      }
      auto step = [&](auto kk_c) __attribute__((always_inline)) {
        constexpr int kk = decltype(kk_c)::value;
        constexpr int src = kk & 1, dst = src ^ 1;
        int nl = 0, pre = 0;
        if constexpr (kk == 0) {
          if (MX && (s & 3) == 1) issue_scales(s / 4 + 1);
        }
        if constexpr (kk < kLoadSteps) {
#pragma unroll
          for (int t = 0; t < kSlots; ++t) {
            if (t / kLoadsPerStep != kk || !used(t)) continue;
            if constexpr (PIN) {
              if (pre < kMfma) {
                compute(kk_c, src, pre, pre + 1);
                ++pre;
                __builtin_amdgcn_sched_barrier(0);
              }
              issue_load(t, sl);
              __builtin_amdgcn_sched_barrier(0);
            } else {
              issue_load(t, sl);
              ++nl;
            }
          }
        }
        if constexpr (kk < 3) {
          read_frags(s, kk + 1, dst);
          if constexpr (kk == 1) read_scales(s + 1);
          compute(kk_c, src, pre, kMfma);
          interleave(kMfma - pre, kk == 1 && MX ? 2 * kReads : kReads, nl);
        } else {
          compute(kk_c, src, 0, kSplit);
          interleave(kSplit, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
          wait_vmcnt<kInFlight>();   // own loads of stage s + 1 landed
          wait_lgkmcnt0();           // own reads of stage s done
          block_barrier();           // ... everyone's
          read_frags(s + 1, 0, dst);
          compute(kk_c, src, kSplit, kMfma);
          interleave(kMfma - kSplit, kReads, 0);
        }
      };
      step(std::integral_constant<int, 0>());
      step(std::integral_constant<int, 1>());
      step(std::integral_constant<int, 2>());
      step(std::integral_constant<int, 3>());
    }
  };
  if constexpr (TAIL && TM == 4) {
    switch (used_blocks) {
      case 1: main_loop(std::integral_constant<int, 1>()); break;
      case 2: main_loop(std::integral_constant<int, 2>()); break;
      case 3: main_loop(std::integral_constant<int, 3>()); break;
      default: main_loop(std::integral_constant<int, 4>()); break;
    }
  } else if constexpr (TAIL && TM == 2) {
    if (used_blocks == 1) main_loop(std::integral_constant<int, 1>());
    else main_loop(std::integral_constant<int, 2>());
  } else {
    main_loop(std::integral_constant<int, TM>());
  }

  // Epilogue.  Every outstanding load (all past the last stage) lands before
  // LDS is reused, and every wave is done reading; then each wave transposes
  // kEpiRows rows of its part at a time through LDS, so that a lane holds 4
  // consecutive columns of one row.
  wait_vmcnt<0>();
  wait_lgkmcnt0();
  block_barrier();
  uint8_t* const stage_out = smem + wave * kEpiWave;
  // row of C behind row r that this wave stages in a pass
  auto row_of = [&](int pass, int r) -> int {
    const int i = pass * (kEpiRows / 32) + r / 32;
    return tile.row0 + (partial ? i * WM + wm : wm * TM + i) * 32 + r % 32;
  };
  const int wcol0 = n0 + wn * WTN;
#pragma unroll
  for (int pass = 0; pass < WTM / kEpiRows; ++pass) {
    if (pass * (kEpiRows / 32) >= used_blocks) break;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int rg = i * 32 + 8 * (e >> 2);
          if (rg / kEpiRows != pass) continue;
          const int r = rg - pass * kEpiRows + 4 * fh + (e & 3);
          const auto v = acc[i][j][e];
          *(uint32_t*)(stage_out + r * kEpiPitch + (j * 32 + fr) * 4) = __builtin_bit_cast(uint32_t, v);
        }
    wait_lgkmcnt0();   // this wave's LDS writes done
    float rs_lane = 0.f;
    uint64_t absent = 0;   // rows of the pass that have no row of A, as bits
    if (KIND == KIND_I8_DEQUANT || gather) {
      const int row = lane < kEpiRows ? row_of(pass, lane) : tile.row_end;
      const int r = a_row_of(p, row, tile.row_end);
      absent = __ballot(r < 0 && row < tile.row_end);
      if (KIND == KIND_I8_DEQUANT && r >= 0) rs_lane = p.row_scale[r];
    }
    // the staged rows, COLS consecutive columns per lane (16 bytes of C: 4 of
    // binary32, 8 of a 16-bit type)
    auto store_rows = [&](auto cols_c) __attribute__((always_inline)) {
      constexpr int COLS = decltype(cols_c)::value;
      constexpr int kLanesPerRow = WTN / COLS;
      constexpr int kRowsPerStore = 64 / kLanesPerRow;
      const int c = (lane % kLanesPerRow) * COLS, col0 = wcol0 + c;
      const bool whole = col0 + COLS <= p.N && p.N % COLS == 0;
      float cs[COLS] = {};
      if constexpr (KIND == KIND_I8_DEQUANT) {
#pragma unroll
        for (int x = 0; x < COLS; ++x)
          if (col0 + x < p.N) cs[x] = p.col_scale[(size_t)tile.group * p.N + col0 + x];
      }
#pragma unroll
      for (int r0 = 0; r0 < kEpiRows; r0 += kRowsPerStore) {
        const int r = r0 + lane / kLanesPerRow;
        float v[COLS];
#pragma unroll
        for (int q = 0; q < COLS / 4; ++q) {
          const i32x4 raw = *(const i32x4*)(stage_out + r * kEpiPitch + (c + 4 * q) * 4);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int bits = raw[x];
            if constexpr (KIND == KIND_I8_DEQUANT) v[4 * q + x] = (float)bits;
            else v[4 * q + x] = __builtin_bit_cast(float, bits);
          }
        }
        if constexpr (KIND == KIND_I8_DEQUANT) {
          const float rs = __shfl(rs_lane, r);
#pragma unroll
          for (int x = 0; x < COLS; ++x) v[x] = (v[x] * rs) * cs[x];
        }
        const int row = row_of(pass, r);
        if (row < tile.row_end) {
          const size_t idx = (size_t)row * p.N + col0;
          if (whole) {
            store16<COLS>(p, idx, v);
          } else {
#pragma unroll
            for (int x = 0; x < COLS; ++x)
              if (col0 + x < p.N) store1(p, idx + x, v[x]);
          }
        }
      }
    };
    if (p.out_type == 0) store_rows(std::integral_constant<int, 4>());
    else store_rows(std::integral_constant<int, 8>());
    // zeros of A times an infinite or NaN weight or scale are not zero: rows
    // without a row of A are written again, once the stores above are done (a
    // select in front of every store takes 1 to 2% of the time)
    if (absent != 0) {
      wait_vmcnt<0>();
      for (uint64_t left = absent; left != 0; left &= left - 1) {
        const size_t idx = (size_t)row_of(pass, __builtin_ctzll(left)) * p.N;
        for (int col = wcol0 + lane; col < min(wcol0 + WTN, p.N); col += 64) store1(p, idx + col, 0.f);
      }
    }
    wait_lgkmcnt0();   // reads done before the next pass overwrites them
  }
}

// ---------------------------------------------------------------------------
// Few rows per group: a workgroup owns 32 columns of C for up to 32 rows, its
// waves split K into runs of 128-byte blocks, and each streams its own run
// through a private ring of DEPTH blocks in LDS (no barrier until the end):
// 32 rows of weights (four 1 KiB loads) and the 8 AG rows of A that the tile
// can have.  The partial sums meet in LDS and are added in wave order, so the
// result does not depend on timing.
//
// Bound by the weights' stream from HBM; the ring keeps WAVES x (DEPTH - 1) x
// 4 KiB of it in flight per workgroup (int8, 8 of 64 experts of 2048 x 4096 on
// one token 12.2 us, 5.5 TB/s; MXFP4, 16 rows of 14336 x 4096 8.8 us, 3.7).
template <int KIND, int WAVES, int DEPTH, int AG>
__global__ __launch_bounds__(WAVES * 64) void grouped_skinny(GroupedArgs p) {
  using Acc = typename GroupedAcc<KIND>::type;
  constexpr bool MX = KIND == KIND_MXFP4;
  constexpr int MT = 8 * AG;
  constexpr int kPitch = 33;
  constexpr int kB = 4096, kA = AG * 1024;
  constexpr int kScB = MX ? 256 : 0, kScA = MX ? 256 : 0;   // 32 rows x 8 bytes each
  constexpr int kBlock = kB + kA + kScB + kScA;
  constexpr int kWaveLds = DEPTH * kBlock;
  static_assert(kWaveLds >= MT * kPitch * 4, "the partial sums reuse the wave's region");
  static_assert(WAVES * kWaveLds <= 160 * 1024, "LDS");
  constexpr int kLoads = 4 + AG + (MX ? 2 : 0);   // per block
  static_assert(kLoads * DEPTH <= 63, "vmcnt range");
  static_assert(DEPTH == 2 || DEPTH == 3, "the waits of the last blocks");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[WAVES * kWaveLds];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const GroupTile tile = find_tile<MT>(p, blockIdx.x);
  if (tile.none) return;
  const int n0 = tile.tn * p.tile_w;
  const int cols = min(p.tile_w, p.N - n0);
  const size_t brow0 = (size_t)tile.group * p.N + n0;
  const bool gather = p.row_index != nullptr;
  const size_t arow0 = gather ? 0 : tile.row0;
  const int arows = gather ? p.a_rows : tile.row_end - tile.row0;
  const uint32_t row_bytes = (uint32_t)p.row_bytes;
  const i32x4 rsrc_a = make_rsrc(p.A + arow0 * row_bytes, (uint32_t)arows * row_bytes);
  const i32x4 rsrc_b = make_rsrc(p.B + brow0 * row_bytes, (uint32_t)cols * row_bytes);
  const i32x4 rsrc_as = make_rsrc(MX ? p.a_scale + arow0 * p.scale_stride : p.A, MX ? (uint32_t)arows * p.scale_stride : 0);
  const i32x4 rsrc_bs = make_rsrc(MX ? p.b_scale + brow0 * p.scale_stride : p.B, MX ? (uint32_t)cols * p.scale_stride : 0);
  uint8_t* const my_smem = smem + wave * kWaveLds;
  const uint32_t my_lds = lds_address(my_smem);

  auto source_row = [&](int r) -> int {   // row r of the tile
    return gather ? a_row_of(p, tile.row0 + r, tile.row_end) : (tile.row0 + r < tile.row_end ? r : -1);
  };
  // copy t of a block: rows 8 t + lane / 8, the chunk whose swizzled position
  // is lane % 8
  uint32_t b_off[4], b_col[4], a_off[AG], a_col[AG];
  uint64_t absent[AG];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int r = 8 * t + lane / 8;
    b_col[t] = swizzle_chunk(r, lane & 7) * 16;
    b_off[t] = (uint32_t)r * row_bytes + b_col[t];
  }
#pragma unroll
  for (int t = 0; t < AG; ++t) {
    const int r = 8 * t + lane / 8;
    const int src = source_row(r);
    a_col[t] = swizzle_chunk(r, lane & 7) * 16;
    a_off[t] = src < 0 ? kOutOfRange : (uint32_t)src * row_bytes + a_col[t];
    // bit 8 x: row 8 t + x has no row of A
    absent[t] = __ballot(src < 0);
  }
  // scales: lane l fetches word l % 2 of row l / 2
  uint32_t bs_off = 0, as_off = kOutOfRange;
  if constexpr (MX) {
    bs_off = (uint32_t)(lane / 2) * (uint32_t)p.scale_stride + (lane & 1) * 4;
    const int src = lane / 2 < MT ? source_row(lane / 2) : -1;
    if (src >= 0) as_off = (uint32_t)src * (uint32_t)p.scale_stride + (lane & 1) * 4;
  }

  const int nblk = p.k_stages;
  const int b0 = (int)((int64_t)nblk * wave / WAVES);
  const int count = (int)((int64_t)nblk * (wave + 1) / WAVES) - b0;
  const int blocks = p.row_bytes / 16;   // MXFP4 blocks

  auto issue = [&](int i) __attribute__((always_inline)) {
    const uint32_t to = my_lds + (i % DEPTH) * kBlock;
    const uint32_t kbyte = (uint32_t)(b0 + i) * 128;
#pragma unroll
    for (int t = 0; t < 4; ++t)
      lds_dma_16<1>(rsrc_b, to + t * 1024, kbyte + b_col[t] < row_bytes ? b_off[t] + kbyte : kOutOfRange);
#pragma unroll
    for (int t = 0; t < AG; ++t)
      lds_dma_16(rsrc_a, to + kB + t * 1024, kbyte + a_col[t] < row_bytes ? a_off[t] + kbyte : kOutOfRange);
    if constexpr (MX) {
      const uint32_t sbyte = (uint32_t)(b0 + i) * 8;   // inside the padded row
      lds_dma_4(rsrc_bs, to + kB + kA, bs_off + sbyte);
      lds_dma_4(rsrc_as, to + kB + kA + kScB, as_off + sbyte);
    }
  };

  const int fr = lane & 31, fh = lane >> 5;
  const int far = fr % MT;   // rows past the tile's repeat its first ones; their results are not stored
  Acc acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0;
  auto contract = [&](int i) __attribute__((always_inline)) {
    const uint8_t* const from = my_smem + (i % DEPTH) * kBlock;
    i32x4 fa[4], fb[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      fb[q] = *(const i32x4*)(from + fr * 128 + (swizzle_chunk(fr, 4 * fh + q) << 4));
      fa[q] = *(const i32x4*)(from + kB + far * 128 + (swizzle_chunk(far, 4 * fh + q) << 4));
    }
    int sa = 0, sb = 0;
    if constexpr (MX) {
      const int mask = scale_mask(b0 + i, fh, blocks);
      sb = *(const int*)(from + kB + kA + fr * 8 + fh * 4) & mask;
      sa = *(const int*)(from + kB + kA + kScB + far * 8 + fh * 4) & mask;
    }
    acc = grouped_mfma<KIND, 0>(fa[0], fb[0], acc, sa, sb);
    acc = grouped_mfma<KIND, 1>(fa[1], fb[1], acc, sa, sb);
    acc = grouped_mfma<KIND, 2>(fa[2], fb[2], acc, sa, sb);
    acc = grouped_mfma<KIND, 3>(fa[3], fb[3], acc, sa, sb);
  };

#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i)
    if (i < count) issue(i);
  int i = 0;
  for (; i + DEPTH - 1 < count; ++i) {
    wait_lgkmcnt0();   // the fragment reads of block i - 1, whose place is taken now
    issue(i + DEPTH - 1);
    wait_vmcnt<(DEPTH - 1) * kLoads>();
    contract(i);
  }
  // the last blocks: nothing more to issue
#pragma unroll
  for (int left = DEPTH - 1; left >= 1; --left) {
    if (count - i == left) {
      if (left == 1) wait_vmcnt<0>();
      else wait_vmcnt<kLoads>();
      contract(i);
      ++i;
    }
  }

  // partial sums: element e of lane l is row 8 (e / 4) + 4 (l / 32) + e % 4,
  // column l % 32
  wait_lgkmcnt0();
  uint32_t* const part = (uint32_t*)my_smem;
#pragma unroll
  for (int e = 0; e < 4 * AG; ++e) {
    const auto v = acc[e];
    part[(8 * (e >> 2) + 4 * fh + (e & 3)) * kPitch + fr] = __builtin_bit_cast(uint32_t, v);
  }
  __syncthreads();
  const uint32_t* const all = (const uint32_t*)smem;
  const int rows = tile.row_end - tile.row0;
  static_assert(WAVES == 4, "each step of the loop below stores 8 rows");
#pragma unroll
  for (int t = 0; t < AG; ++t) {
    const int r = 8 * t + tid / 32, c = tid % 32;
    if (r >= rows || c >= cols) continue;
    float v;
    if constexpr (KIND == KIND_I8_DEQUANT) {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) sum += (int)all[w * (kWaveLds / 4) + r * kPitch + c];
      const int src = a_row_of(p, tile.row0 + r, tile.row_end);
      const float rs = src < 0 ? 0.f : p.row_scale[src];
      v = ((float)sum * rs) * p.col_scale[(size_t)tile.group * p.N + n0 + c];
    } else {
      v = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) v += __builtin_bit_cast(float, all[w * (kWaveLds / 4) + r * kPitch + c]);
    }
    // (zeros of A times an infinite or NaN weight or scale are not zero)
    if ((absent[t] >> (8 * (tid / 32))) & 1) v = 0.f;
    store1(p, (size_t)(tile.row0 + r) * p.N + n0 + c, v);
  }
}

}  // namespace lpgemm
