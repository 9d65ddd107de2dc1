// gated_two_group.hip -- launches of the two-group kernel
// (grouped_two_group.hpp): the gated product and its gradient with B
// K-contiguous.
#include "grouped_two_group.hpp"

namespace tla {

int launch_gated_two_group_nk(const GroupedParams& p, int type, int role, hipStream_t s) {
  if (role == kGated)
    return type == TLA_BF16 ? launch<kBF16, kNK, kGated>(p, s) : launch<kF16, kNK, kGated>(p, s);
  return type == TLA_BF16 ? launch<kBF16, kNK, kGateGrad>(p, s) : launch<kF16, kNK, kGateGrad>(p, s);
}

}  // namespace tla
