// gated_two_group_grad_kn.hip -- launches of the two-group kernel
// (grouped_two_group.hpp): the gated product's gradient with 16-bit [K, N] weights.
#include "grouped_two_group.hpp"

namespace tla {

int launch_two_group_grad_kn(const GroupedParams& p, int type, hipStream_t s) {
  return type == TLA_BF16 ? launch_act<kBF16, kKN, kGateGrad>(p, s) : launch_act<kF16, kKN, kGateGrad>(p, s);
}

}  // namespace tla
