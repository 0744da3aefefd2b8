// Products of many rows with 4-bit weights, bf16, groups of 32.
#define LPGEMM_W4_DEFINE
#include "w4_tile.hpp"

namespace lpgemm {
template lpgemm_status run_w4_tile<TypeBF16, 1>(const W4Plan&, W4TileArgs, hipStream_t);
}
