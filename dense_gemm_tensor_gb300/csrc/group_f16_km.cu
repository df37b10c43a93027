// f16: grouped products with K-major weights.
#include "group_launch.h"

namespace dgt {
DGT_DEFINE_GROUP(f16_km, KIND_F16, GROUP_W_K)
}  // namespace dgt
