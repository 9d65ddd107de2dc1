// grouped_two_group_rows.hip -- launches of the two-group kernel
// (grouped_two_group.hpp): the forms whose slabs are rows of
// k: the product with 16-bit [K, N] weights and the weight gradient.
#include "grouped_two_group.hpp"

namespace tla {

int launch_two_group_kn(const GroupedParams& p, int type, hipStream_t s) {
  return type == TLA_BF16 ? launch<kBF16, kKN>(p, s) : launch<kF16, kKN>(p, s);
}

int launch_wgrad_two_group(const GroupedParams& p, int type, hipStream_t s) {
  return type == TLA_BF16 ? launch<kBF16, kGrad>(p, s) : launch<kF16, kGrad>(p, s);
}

}  // namespace tla
