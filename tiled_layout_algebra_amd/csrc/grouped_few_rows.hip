// grouped_few_rows.hip -- launches of the kernel for few rows
// (grouped_few_rows.hpp): the grouped products.
#include "grouped_few_rows.hpp"

namespace tla {
namespace {

template <int kCode>
int pick(const GroupedParams& p, int mt, hipStream_t s) {
  const bool narrow = few_rows_narrow(p.rows, p.groups, p.N);
  if (mt == 1) return narrow ? launch<kCode, 1, 1, 8>(p, s) : launch<kCode, 1, 2, 4>(p, s);
  if (mt == 2) return narrow ? launch<kCode, 2, 1, 8>(p, s) : launch<kCode, 2, 2, 4>(p, s);
  return narrow ? launch<kCode, 4, 1, 8>(p, s) : launch<kCode, 4, 2, 4>(p, s);
}

}  // namespace

int launch_grouped_few_rows(const GroupedParams& p, int type, int mt, hipStream_t s) {
  switch (type) {
    case TLA_BF16: return pick<kBF16>(p, mt, s);
    case TLA_F16: return pick<kF16>(p, mt, s);
    case TLA_E4M3: return pick<kE4M3>(p, mt, s);
    case TLA_I8: return pick<kI8>(p, mt, s);
    default: return TLA_ERR_UNSUPPORTED;
  }
}

}  // namespace tla
