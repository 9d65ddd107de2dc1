// grouped_general.hip -- launches of the register-staged kernel
// (grouped_general.hpp): the products and the weight gradient.
#include "grouped_general.hpp"

namespace tla {
namespace {

template <int kCode, int kBView, bool kWgrad>
int launch(const GroupedParams& p, hipStream_t stream) {
  if constexpr (kBView != kBElem) {
    constexpr int kCE = 16 / type_bytes(kCode);
    // the lines: of K (A, or both), of N, of both extents of the gradient
    const bool a_long = kWgrad ? p.M >= kCE : p.K >= kCE;
    const bool b_long = kBView == kBKc ? p.K >= kCE : p.N >= kCE;
    if (a_long && b_long) return launch_form<kCode, kBView, kWgrad, true>(p, stream);
  }
  return launch_form<kCode, kBView, kWgrad, false>(p, stream);
}

}  // namespace

int launch_grouped_general(const GroupedParams& p, int type, bool b_kc, hipStream_t s) {
  switch (type) {
    case TLA_BF16:
      return b_kc ? launch<kBF16, kBKc, false>(p, s) : launch<kBF16, kBRows, false>(p, s);
    case TLA_F16:
      return b_kc ? launch<kF16, kBKc, false>(p, s) : launch<kF16, kBRows, false>(p, s);
    case TLA_E4M3:
      return b_kc ? launch<kE4M3, kBKc, false>(p, s) : launch<kE4M3, kBElem, false>(p, s);
    case TLA_I8:
      return b_kc ? launch<kI8, kBKc, false>(p, s) : launch<kI8, kBElem, false>(p, s);
    default: return TLA_ERR_UNSUPPORTED;
  }
}

int launch_wgrad_general(const GroupedParams& p, int type, hipStream_t s) {
  switch (type) {
    case TLA_BF16: return launch<kBF16, kBRows, true>(p, s);
    case TLA_F16: return launch<kF16, kBRows, true>(p, s);
    default: return TLA_ERR_UNSUPPORTED;
  }
}

}  // namespace tla
