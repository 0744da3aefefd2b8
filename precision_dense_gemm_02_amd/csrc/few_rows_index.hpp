// Where few_rows (few_rows_kernels.hpp) loads the scales of 4-bit weights and
// the rows of X that it copies into LDS: plain arithmetic, in a file of its own
// for the host's tests.
#pragma once

namespace lpgemm {

// A wave takes runs of two blocks of 128 k.  The scales of a run's groups come
// as one load (w4 = 1: two, one per block) per 16 weight rows: 16 rows by the
// groups that the lane rows q = 0 .. 3 hold, counted from the load's first one.
// w4: K-steps of 32 that share a scale, 4 for groups of 128 and more, of which
// group_shift is the log2 of a group's blocks.
constexpr int kScaleRun = 2;
constexpr int scale_loads(int w4) { return w4 == 1 ? 2 : 1; }

// The first group of load t of a run.
constexpr int scale_first_group(int w4, int group_shift, int run, int t) {
  return w4 == 4   ? (run * kScaleRun) >> group_shift
         : w4 == 2 ? run * 4
                   : (run * kScaleRun + t) * 4;
}
// The group that lane row q holds, from the load's first (w4 = 4: one per block).
constexpr int scale_lane_group(int w4, int group_shift, int q) { return w4 == 4 ? (q & 1) >> group_shift : q; }

// The last run of an odd number of whole blocks has no second block, whose
// groups would lie behind their row's last and, in the last row, behind the
// scales.  Whether the load has a block at all (w4 = 1: load t is block t's) ...
constexpr bool scale_load_there(int w4, int run, int t, int whole) { return run * kScaleRun + (w4 == 1 ? t : 0) < whole; }
// ... and whether lane row q's group is that of the run's second block, and is
// loaded only where that block is there.
constexpr bool scale_second_block(int w4, int q) { return w4 == 4 ? (q & 1) != 0 : w4 == 2 && q >= 2; }

// The row of X that 16-byte chunk i of rows of `chunks` is in (K = 0: there are
// none, and none is copied).
constexpr int x_chunk_row(int i, int chunks) { return chunks > 0 ? i / chunks : 0; }

}  // namespace lpgemm
