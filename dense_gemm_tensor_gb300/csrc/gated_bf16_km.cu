#include "group_launch.h"

namespace dgt {
DGT_DEFINE_GATED(bf16_km, KIND_BF16, GROUP_W_K)
}  // namespace dgt
