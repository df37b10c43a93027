#include "group_launch.h"

namespace dgt {
DGT_DEFINE_GATED(f16_rm, KIND_F16, GROUP_W_MN)
}  // namespace dgt
