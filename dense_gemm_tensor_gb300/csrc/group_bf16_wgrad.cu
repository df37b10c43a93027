// bf16: the grouped products' weight gradient.
#include "group_launch.h"

namespace dgt {
DGT_DEFINE_GROUP_WGRAD(bf16_wgrad, KIND_BF16)
}  // namespace dgt
