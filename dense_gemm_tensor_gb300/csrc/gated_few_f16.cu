// f16: the dense gated product of few rows.
#include "gated_few.h"

namespace dgt {
DGT_DEFINE_GATED_FEW(f16, KIND_F16)
}  // namespace dgt
