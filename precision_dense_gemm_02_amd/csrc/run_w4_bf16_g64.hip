// Products of many rows with 4-bit weights, bf16, groups of 64.
#define LPGEMM_W4_DEFINE
#include "w4_tile.hpp"

namespace lpgemm {
template lpgemm_status run_w4_tile<TypeBF16, 2>(const W4Plan&, W4TileArgs, hipStream_t);
}
