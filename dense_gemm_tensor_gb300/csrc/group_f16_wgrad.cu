// f16: the grouped products' weight gradient.
#include "group_launch.h"

namespace dgt {
DGT_DEFINE_GROUP_WGRAD(f16_wgrad, KIND_F16)
}  // namespace dgt
