// Products of many rows with 4-bit weights, f16, groups of 128 and more.
#define LPGEMM_W4_DEFINE
#include "w4_tile.hpp"

namespace lpgemm {
template lpgemm_status run_w4_tile<TypeF16, 4>(const W4Plan&, W4TileArgs, hipStream_t);
}
