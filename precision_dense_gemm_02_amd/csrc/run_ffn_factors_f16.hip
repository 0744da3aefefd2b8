// Products with 4-bit weights written out in 16 bits, f16.
#define LPGEMM_FFN_DEFINE
#include "ffn.hpp"

namespace lpgemm {
template lpgemm_status run_tile<TypeF16, true>(int, TileArgs, float*, int64_t, int, hipStream_t);
}
