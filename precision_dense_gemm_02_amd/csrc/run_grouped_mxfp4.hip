// The grouped kernels for MXFP4 operands: run_grouped<KIND_MXFP4>.
#define LPGEMM_GROUPED_DEFINE
#include "grouped.hpp"

namespace lpgemm {
template lpgemm_status run_grouped<KIND_MXFP4>(GroupedArgs, int, hipStream_t);
}  // namespace lpgemm
