// two_group_lds.hpp -- how the two-group kernel (grouped_two_group.hpp) divides its
// LDS: two A slots, three B slots, and the waves' epilogue regions over them.
// Plain C++, so that the layout is checked without a GPU.
#pragma once

namespace tla {

constexpr int kTwoGroupSlab = 256 * 128;         // one operand, one k-tile
constexpr int kTwoGroupB = 2 * kTwoGroupSlab;    // [A0 A1 | B0 B1 B2]
constexpr int kTwoGroupLds = 5 * kTwoGroupSlab;  // of the workgroup

// First byte of wave w's epilogue region of `bytes` bytes, KT k-tiles behind it.
// Group 0 (waves 0 .. 3) passes a barrier after its last fragment reads, and A's
// slots are read by nobody from then on.  Group 1 goes from its last MFMAs into
// its epilogue without one.  late: these MFMAs still have fragments of B read
// between them, from slot (KT - 1) % 3, so a wave that is done first must not write
// there: group 1's regions are then the two other B slots.
constexpr int two_group_region(int w, int bytes, bool late, int KT) {
  if (!late || w < 4) return w * bytes;
  return kTwoGroupB + (KT + (w >> 1 & 1)) % 3 * kTwoGroupSlab + (w & 1) * (kTwoGroupSlab / 2);
}

}  // namespace tla
