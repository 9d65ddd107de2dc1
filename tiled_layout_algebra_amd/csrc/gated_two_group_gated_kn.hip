// gated_two_group_gated_kn.hip -- launches of the two-group kernel
// (grouped_two_group.hpp): the gated product with 16-bit [K, N] weights.
#include "grouped_two_group.hpp"

namespace tla {

int launch_two_group_gated_kn(const GroupedParams& p, int type, hipStream_t s) {
  return type == TLA_BF16 ? launch_act<kBF16, kKN, kGated>(p, s) : launch_act<kF16, kKN, kGated>(p, s);
}

}  // namespace tla
