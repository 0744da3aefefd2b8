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

// The bytes of `rows` weight rows' scales from the load's first group on: the
// records of its descriptor.  The last run of an odd number of whole blocks has
// no second block: its lanes reach past their row's last group, into the next
// row's or, behind the last row, past the records, where a load gives 0.
constexpr int scale_records(int rows, int groups, int first_group) {
  return rows * groups > first_group ? 2 * (rows * groups - first_group) : 0;
}

// The row of X that 16-byte chunk i of rows of `chunks` is in (K = 0: there are
// none, and none is copied).
constexpr int x_chunk_row(int i, int chunks) { return chunks > 0 ? i / chunks : 0; }

}  // namespace lpgemm
