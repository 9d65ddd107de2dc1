// gated_two_group_rows.hip -- launches of the two-group kernel
// (grouped_two_group.hpp): the gated product and its gradient with 16-bit [K, N]
// weights.
#include "grouped_two_group.hpp"

namespace tla {

int launch_gated_two_group_kn(const GroupedParams& p, int type, int role, hipStream_t s) {
  if (role == kGated)
    return type == TLA_BF16 ? launch<kBF16, kKN, kGated>(p, s) : launch<kF16, kKN, kGated>(p, s);
  return type == TLA_BF16 ? launch<kBF16, kKN, kGateGrad>(p, s) : launch<kF16, kKN, kGateGrad>(p, s);
}

}  // namespace tla
