// grouped_two_group_8bit.hip -- launches of the two-group kernel
// (grouped_two_group.hpp): the product of 8-bit operands.
#include "grouped_two_group.hpp"

namespace tla {

int launch_two_group_nk8(const GroupedParams& p, int type, hipStream_t s) {
  return type == TLA_I8 ? launch<kI8, kNK>(p, s) : launch<kE4M3, kNK>(p, s);
}

}  // namespace tla
