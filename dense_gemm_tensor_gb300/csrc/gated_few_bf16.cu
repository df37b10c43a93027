// bf16: the dense gated product of few rows.
#include "gated_few.h"

namespace dgt {
DGT_DEFINE_GATED_FEW(bf16, KIND_BF16)
}  // namespace dgt
