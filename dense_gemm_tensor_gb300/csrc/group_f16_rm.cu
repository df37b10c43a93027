// f16: grouped products with row-major weights.
#include "group_launch.h"

namespace dgt {
DGT_DEFINE_GROUP(f16_rm, KIND_F16, GROUP_W_MN)
}  // namespace dgt
