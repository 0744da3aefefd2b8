// Products of the gated feed-forward block, f16 operands.
#define LPGEMM_FFN_DEFINE
#include "ffn.hpp"

namespace lpgemm {
template lpgemm_status run_tile<TypeF16, false>(int, TileArgs, float*, int64_t, int, hipStream_t);
}
