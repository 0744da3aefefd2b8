// The grouped kernels for binary16 operands: run_grouped<KIND_F16>.
#define LPGEMM_GROUPED_DEFINE
#include "grouped.hpp"

namespace lpgemm {
template lpgemm_status run_grouped<KIND_F16>(GroupedArgs, int, hipStream_t);
}  // namespace lpgemm
