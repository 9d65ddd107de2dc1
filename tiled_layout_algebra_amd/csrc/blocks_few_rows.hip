// blocks_few_rows.hip -- launches of the kernel for few rows
// (grouped_few_rows.hpp): e4m3 with block scales, plain and gated.  Bound by the weights'
// way from memory (figures there).
#include "grouped_few_rows.hpp"

namespace tla {
namespace {

int plain(const GroupedParams& p, int mt, hipStream_t s) {
  if (few_rows_narrow(p.rows, p.groups, p.N)) {
    if (mt == 1) return launch<kE4M3Blocks, 1, 1, 8>(p, s);
    if (mt == 2) return launch<kE4M3Blocks, 2, 1, 8>(p, s);
    return launch<kE4M3Blocks, 4, 1, 8>(p, s);
  }
  if (mt == 1) return launch<kE4M3Blocks, 1, 2, 4>(p, s);
  if (mt == 2) return launch<kE4M3Blocks, 2, 2, 4>(p, s);
  return launch<kE4M3Blocks, 4, 2, 4>(p, s);
}

int gated_product(const GroupedParams& p, int mt, hipStream_t s) {
  if (mt == 1) return launch<kE4M3Blocks, 1, 2, 8, kGated>(p, s);
  if (mt == 2) return launch<kE4M3Blocks, 2, 2, 8, kGated>(p, s);
  return launch<kE4M3Blocks, 4, 2, 4, kGated>(p, s);
}

}  // namespace

int launch_blocks_few_rows(const GroupedParams& p, int mt, bool gated, hipStream_t s) {
  return gated ? gated_product(p, mt, s) : plain(p, mt, s);
}

}  // namespace tla
