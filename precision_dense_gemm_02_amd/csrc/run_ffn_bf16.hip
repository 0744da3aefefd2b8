// Products of the gated feed-forward block, bf16 operands.
#define LPGEMM_FFN_DEFINE
#include "ffn.hpp"

namespace lpgemm {
template lpgemm_status run_tile<TypeBF16, false>(int, TileArgs, float*, int64_t, int, hipStream_t);
}
