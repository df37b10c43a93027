// bf16: grouped products with K-major weights.
#include "group_launch.h"

namespace dgt {
DGT_DEFINE_GROUP(bf16_km, KIND_BF16, GROUP_W_K)
}  // namespace dgt
