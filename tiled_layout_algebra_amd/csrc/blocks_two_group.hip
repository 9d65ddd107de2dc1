// blocks_two_group.hip -- launches of the two-group kernel
// (grouped_two_group.hpp): e4m3 with block scales, plain and gated.
#include "grouped_two_group.hpp"

namespace tla {

int launch_blocks_two_group(const GroupedParams& p, bool gated, hipStream_t s) {
  return gated ? launch_act<kE4M3Blocks, kNK, kGated>(p, s) : launch_act<kE4M3Blocks, kNK, kPlain>(p, s);
}

}  // namespace tla
