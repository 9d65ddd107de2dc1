// gated_two_group_grad_nk.hip -- launches of the two-group kernel
// (grouped_two_group.hpp): the gated product's gradient with B K-contiguous.
#include "grouped_two_group.hpp"

namespace tla {

int launch_two_group_grad_nk(const GroupedParams& p, int type, hipStream_t s) {
  return type == TLA_BF16 ? launch_act<kBF16, kNK, kGateGrad>(p, s) : launch_act<kF16, kNK, kGateGrad>(p, s);
}

}  // namespace tla
