// bf16: grouped products with row-major weights.
#include "group_launch.h"

namespace dgt {
DGT_DEFINE_GROUP(bf16_rm, KIND_BF16, GROUP_W_MN)
}  // namespace dgt
