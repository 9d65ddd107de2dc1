// grouped_two_group_shift.hip -- launches of the two-group kernel
// (grouped_two_group.hpp): the product of operands at any byte address with B
// K-contiguous.
#include "grouped_two_group.hpp"

namespace tla {

int launch_two_group_shift(const GroupedParams& p, int type, hipStream_t s) {
  switch (type) {
    case TLA_BF16: return launch<kBF16, kNKShift>(p, s);
    case TLA_F16: return launch<kF16, kNKShift>(p, s);
    case TLA_E4M3: return launch<kE4M3, kNKShift>(p, s);
    case TLA_I8: return launch<kI8, kNKShift>(p, s);
    default: return TLA_ERR_UNSUPPORTED;
  }
}

}  // namespace tla
