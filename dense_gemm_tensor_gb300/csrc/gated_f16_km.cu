#include "group_launch.h"

namespace dgt {
DGT_DEFINE_GATED(f16_km, KIND_F16, GROUP_W_K)
}  // namespace dgt
