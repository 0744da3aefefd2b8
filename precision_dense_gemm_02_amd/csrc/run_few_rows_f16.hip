// Products of few rows, f16 operands.
#define LPGEMM_FEW_ROWS_DEFINE
#include "few_rows.hpp"

namespace lpgemm {
template lpgemm_status run_few_rows<TypeF16>(const FewRowsArgs&, int, int, hipStream_t);
}
