// gated_two_group_gated_nk.hip -- launches of the two-group kernel
// (grouped_two_group.hpp): the gated product with B K-contiguous.
#include "grouped_two_group.hpp"

namespace tla {

int launch_two_group_gated_nk(const GroupedParams& p, int type, hipStream_t s) {
  return type == TLA_BF16 ? launch_act<kBF16, kNK, kGated>(p, s) : launch_act<kF16, kNK, kGated>(p, s);
}

}  // namespace tla
