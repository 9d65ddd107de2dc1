// grouped_two_group.hip -- launches of the two-group kernel
// (grouped_two_group.hpp): the product of 16-bit operands
// with B K-contiguous.
#include "grouped_two_group.hpp"

namespace tla {

int launch_two_group_nk16(const GroupedParams& p, int type, hipStream_t s) {
  return type == TLA_BF16 ? launch<kBF16, kNK>(p, s) : launch<kF16, kNK>(p, s);
}

}  // namespace tla
