#include "group_launch.h"

namespace dgt {
DGT_DEFINE_GATED(bf16_rm, KIND_BF16, GROUP_W_MN)
}  // namespace dgt
