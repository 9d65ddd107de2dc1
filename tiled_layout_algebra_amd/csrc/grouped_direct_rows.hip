// grouped_direct_rows.hip -- launches of the direct-copy kernel
// (grouped_direct.hpp) whose slabs are rows of k: the product with 16-bit
// [K, N] weights and the weight gradient.
#include "grouped_direct.hpp"

namespace tla {
namespace {

template <int kForm>
int pick(const GroupedParams& p, int type, int shape, hipStream_t s) {
  const bool bf = type == TLA_BF16;
  if (shape == kDirect128x3)
    return bf ? launch<kBF16, kForm, 128, 128, 3, 1, 2, 4>(p, s)
              : launch<kF16, kForm, 128, 128, 3, 1, 2, 4>(p, s);
  return bf ? launch<kBF16, kForm, 128, 128, 2, 1, 2, 2>(p, s)
            : launch<kF16, kForm, 128, 128, 2, 1, 2, 2>(p, s);
}

}  // namespace

int launch_grouped_direct_kn(const GroupedParams& p, int type, int shape, hipStream_t s) {
  return pick<kKN>(p, type, shape, s);
}

int launch_wgrad_direct(const GroupedParams& p, int type, int shape, hipStream_t s) {
  return pick<kGrad>(p, type, shape, s);
}

}  // namespace tla
