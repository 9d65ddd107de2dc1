// grouped_direct_shift.hip -- launches of the direct-copy kernel
// (grouped_direct.hpp) for operands at any byte address with B K-contiguous.
#include "grouped_direct.hpp"

namespace tla {
namespace {

template <int kCode>
int pick(const GroupedParams& p, int shape, hipStream_t s) {
  if (shape == kDirect64x3) return launch<kCode, kNKShift, 64, 128, 3, 1, 2, 2>(p, s);
  return launch<kCode, kNKShift, 128, 128, 3, 1, 2, 4>(p, s);
}

}  // namespace

int launch_grouped_direct_shift(const GroupedParams& p, int type, int shape, hipStream_t s) {
  switch (type) {
    case TLA_BF16: return pick<kBF16>(p, shape, s);
    case TLA_F16: return pick<kF16>(p, shape, s);
    case TLA_E4M3: return pick<kE4M3>(p, shape, s);
    case TLA_I8: return pick<kI8>(p, shape, s);
    default: return TLA_ERR_UNSUPPORTED;
  }
}

}  // namespace tla
