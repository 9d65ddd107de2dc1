// gated_direct.hip -- launches of the direct-copy kernel (grouped_direct.hpp):
// the gated product and its gradient.  Wave tiles are 32 x 64: two 32-column
// MFMA tiles, so that a wave of the gated product holds both sums of an element.
#include "grouped_direct.hpp"

namespace tla {
namespace {

template <int kCode, int kRole>
int pick(const GroupedParams& p, int shape, hipStream_t s) {
  if (shape == kDirect64x3) return launch<kCode, kNK, 64, 128, 3, 1, 2, 2, kRole>(p, s);
  return launch<kCode, kNK, 128, 128, 3, 1, 4, 2, kRole>(p, s);
}

template <int kCode, int kRole>
int pick_kn(const GroupedParams& p, hipStream_t s) {
  return launch<kCode, kKN, 128, 128, 3, 1, 4, 2, kRole>(p, s);
}

}  // namespace

int launch_gated_direct_nk(const GroupedParams& p, int type, int shape, int role, hipStream_t s) {
  if (role == kGated)
    return type == TLA_BF16 ? pick<kBF16, kGated>(p, shape, s) : pick<kF16, kGated>(p, shape, s);
  return type == TLA_BF16 ? pick<kBF16, kGateGrad>(p, shape, s) : pick<kF16, kGateGrad>(p, shape, s);
}

int launch_gated_direct_kn(const GroupedParams& p, int type, int role, hipStream_t s) {
  if (role == kGated)
    return type == TLA_BF16 ? pick_kn<kBF16, kGated>(p, s) : pick_kn<kF16, kGated>(p, s);
  return type == TLA_BF16 ? pick_kn<kBF16, kGateGrad>(p, s) : pick_kn<kF16, kGateGrad>(p, s);
}

}  // namespace tla
