// Products of few rows, bf16 operands.
#define LPGEMM_FEW_ROWS_DEFINE
#include "few_rows.hpp"

namespace lpgemm {
template lpgemm_status run_few_rows<TypeBF16>(const FewRowsArgs&, int, int, hipStream_t);
}
