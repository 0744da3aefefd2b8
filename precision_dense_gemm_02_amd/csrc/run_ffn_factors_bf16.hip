// Products with 4-bit weights written out in 16 bits, bf16.
#define LPGEMM_FFN_DEFINE
#include "ffn.hpp"

namespace lpgemm {
template lpgemm_status run_tile<TypeBF16, true>(int, TileArgs, float*, int64_t, int, hipStream_t);
}
