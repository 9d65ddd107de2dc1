// blocks_two_group.hip -- launches of the two-group kernel
// (grouped_two_group.hpp): e4m3 with block scales, plain and gated.
#include "grouped_two_group.hpp"

namespace tla {

int launch_blocks_two_group(const GroupedParams& p, bool gated, hipStream_t s) {
  return gated ? launch<kE4M3Blocks, kNK, kGated>(p, s) : launch<kE4M3Blocks, kNK>(p, s);
}

}  // namespace tla
