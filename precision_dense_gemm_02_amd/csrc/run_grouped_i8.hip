// The grouped kernels for int8 operands: run_grouped<KIND_I8_DEQUANT>.
#define LPGEMM_GROUPED_DEFINE
#include "grouped.hpp"

namespace lpgemm {
template lpgemm_status run_grouped<KIND_I8_DEQUANT>(GroupedArgs, int, hipStream_t);
}  // namespace lpgemm
