// Walks the loads of the kernel for few rows (csrc/few_rows_index.hpp) as its
// lanes issue them, on the host.
//
//   few_rows_index N K group           the bytes behind the scales that lanes
//                                      would reach if each run had two blocks,
//                                      then those that they reach
//   few_rows_index all                 every size of a sweep: nothing behind the
//                                      scales, and every group that a whole
//                                      block needs loaded by the lane that hands
//                                      it round
//   few_rows_index copy K rows threads how often each chunk of X is copied: the
//                                      least and the most, and chunks besides
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "../precision_dense_gemm_02_amd/csrc/few_rows_index.hpp"

using namespace lpgemm;

namespace {

struct Walk {
  long free_past = 0, past = 0;   // bytes behind the array: with two blocks in every run, as loaded
  bool right = true;
};

bool loaded(int w4, int run, int t, int q, int whole) {
  return scale_load_there(w4, run, t, whole) && (w4 == 1 || run * kScaleRun + 1 < whole || !scale_second_block(w4, q));
}

Walk walk(int N, int K, int group) {
  const int w4 = group == 32 ? 1 : group == 64 ? 2 : 4, shift = group == 256 ? 1 : 0;
  const int groups = K / group, whole = K / 128, runs = (whole + kScaleRun - 1) / kScaleRun;
  const long size = 2l * N * groups;
  Walk out;
  for (int row0 = 0; row0 < N; row0 += 16) {
    const int rows = N - row0 < 16 ? N - row0 : 16;
    for (int run = 0; run < runs; ++run) {
      for (int t = 0; t < scale_loads(w4); ++t) {
        const int first = scale_first_group(w4, shift, run, t);
        const long base = 2l * row0 * groups + 2l * first;
        for (int r = 0; r < rows; ++r)
          for (int q = 0; q < 4; ++q) {
            const long past = base + 2l * (r * groups + scale_lane_group(w4, shift, q)) + 2 - size;
            if (past > out.free_past) out.free_past = past;
            if (loaded(w4, run, t, q, whole) && past > out.past) out.past = past;
          }
      }
      // the groups of the blocks that are there, from the lane rows that hand them round
      for (int h = 0; h < kScaleRun; ++h) {
        const int block = run * kScaleRun + h;
        if (block >= whole) continue;
        for (int t = 0; t < 4 / w4; ++t) {
          const int load = w4 == 1 ? h : 0, from = w4 == 1 ? t : w4 == 2 ? 2 * h + t : h;
          const int first = scale_first_group(w4, shift, run, load);
          const int have = first + scale_lane_group(w4, shift, from), want = (128 * block + 32 * w4 * t) / group;
          if (have != want || !loaded(w4, run, load, from, whole)) out.right = false;
        }
      }
    }
  }
  return out;
}

// The copy of X into LDS: chunks i of every thread, as the kernel takes them.
void copy(int K, int rows, int threads) {
  const int chunks = (K + 127) / 128 * 16, all = rows * chunks;
  std::vector<int> times(all);
  int besides = 0;
  for (int thread = 0; thread < threads; ++thread) {
    auto take = [&](int i) {
      const int row = x_chunk_row(i, chunks), c = i - row * chunks;
      if (i >= all) return;
      if (row < 0 || row >= rows || c < 0 || c >= chunks) ++besides;
      else ++times[row * chunks + c];
    };
    for (int i = 2 * threads + thread; i < all; i += threads) take(i);
    take(thread);
    take(threads + thread);
  }
  int least = all ? times[0] : 0, most = 0;
  for (int n : times) least = n < least ? n : least, most = n > most ? n : most;
  printf("%d %d %d\n", least, most, besides);
}

}  // namespace

int main(int argc, char** argv) {
  if (argc == 5 && strcmp(argv[1], "copy") == 0) {
    copy(atoi(argv[2]), atoi(argv[3]), atoi(argv[4]));
    return 0;
  }
  if (argc == 4) {
    const Walk w = walk(atoi(argv[1]), atoi(argv[2]), atoi(argv[3]));
    printf("%ld %ld %d\n", w.free_past, w.past, w.right);
    return 0;
  }
  if (argc != 2 || strcmp(argv[1], "all") != 0) return 2;
  long sizes = 0, past = 0, wrong = 0, reached = 0;
  for (int group = 32; group <= 256; group *= 2)
    for (int K = group; K <= 4608; K += group)
      for (int N : {1, 2, 15, 16, 17, 31, 32, 33, 100}) {
        const Walk w = walk(N, K, group);
        ++sizes, past += w.past > 0, wrong += !w.right, reached += w.free_past > 0;
      }
  printf("sizes %ld past %ld wrong %ld reached %ld\n", sizes, past, wrong, reached);
}
