// e4m3: grouped products with K-major weights.
#include "group_launch.h"

namespace dgt {
DGT_DEFINE_GROUP(e4m3_km, KIND_E4M3, GROUP_W_K)
}  // namespace dgt
