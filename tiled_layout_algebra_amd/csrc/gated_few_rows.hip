// gated_few_rows.hip -- launches of the kernel for few rows
// (grouped_few_rows.hpp): the gated product in 16 bits.  A workgroup has 16
// columns of both projections.  Bound by the weights' way from memory (figures in
// grouped_few_rows.hpp).
#include "grouped_few_rows.hpp"

namespace tla {
namespace {

template <int kCode>
int pick(const GroupedParams& p, int mt, hipStream_t s) {
  if (mt == 1) return launch<kCode, 1, 2, 8, kGated>(p, s);
  if (mt == 2) return launch<kCode, 2, 2, 8, kGated>(p, s);
  return launch<kCode, 4, 2, 4, kGated>(p, s);
}

}  // namespace

int launch_gated_few_rows(const GroupedParams& p, int type, int mt, hipStream_t s) {
  return type == TLA_BF16 ? pick<kBF16>(p, mt, s) : pick<kF16>(p, mt, s);
}

}  // namespace tla
