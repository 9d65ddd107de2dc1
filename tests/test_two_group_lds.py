"""The two-group kernel's LDS layout on the CPU: no wave's epilogue region meets what
another wave still reads behind the last barrier.

The schedule it is held against (grouped_two_group.hpp): k-tile kt lies in A slot
kt % 2 and B slot kt % 3.  Behind the last barrier group 0 (waves 0 .. 3) is done
reading, and a wave of group 1 still multiplies k-tile KT - 1: with late fragments it
reads that k-tile's B slot meanwhile, with all fragments in registers nothing."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_layout_algebra_amd", "csrc")
SLAB, LDS = 256 * 128, 5 * 256 * 128
TILES = range(1, 20)


def clashes(first, size, late, KT):
    """Pairs of a wave and what its region [first(w), first(w) + size) may overwrite."""
    out = [(w, v) for w in range(8) for v in range(w) if abs(first(w) - first(v)) < size]
    out += [(w, "outside") for w in range(8) if not 0 <= first(w) <= LDS - size]
    if late:
        slot = 2 * SLAB + (KT - 1) % 3 * SLAB
        out += [(w, "the last k-tile's B") for w in range(8) if slot - size < first(w) < slot + SLAB]
    return out


@pytest.fixture(scope="module")
def regions(tmp_path_factory):
    """{(wave, bytes, late, KT): first byte}, from the header that the kernel includes."""
    d = tmp_path_factory.mktemp("lds")
    (d / "a.cpp").write_text('''
#include <cstdio>
#include "two_group_lds.hpp"
static_assert(tla::kTwoGroupSlab == %d && tla::kTwoGroupLds == %d && tla::kTwoGroupB == 2 * %d);
int main() {
  for (int kt = 1; kt < 20; ++kt)
    for (int late = 0; late < 2; ++late)
      for (int bytes = 8192; bytes <= 16384; bytes *= 2)
        for (int w = 0; w < 8; ++w)
          std::printf("%%d %%d %%d %%d %%d\\n", w, bytes, late, kt, tla::two_group_region(w, bytes, late, kt));
}
''' % (SLAB, LDS, SLAB))
    subprocess.run(["g++", "-std=c++20", "-I", CSRC, str(d / "a.cpp"), "-o", str(d / "a")], check=True)
    lines = subprocess.run([str(d / "a")], check=True, capture_output=True, text=True).stdout.split("\n")
    rows = [tuple(map(int, x.split())) for x in lines if x]
    return {r[:4]: r[4] for r in rows}


@pytest.mark.parametrize("late", [0, 1])
@pytest.mark.parametrize("size", [8192, 16384])
def test_regions(regions, size, late):
    for KT in TILES:
        assert not clashes(lambda w: regions[w, size, late, KT], size, late, KT), KT
        assert all(regions[w, size, late, KT] % 1024 == 0 for w in range(8))


def test_the_check_sees_regions_in_wave_order():
    """Regions side by side from 0 on meet the last k-tile's slot for two of three lengths."""
    hit = [KT for KT in TILES if clashes(lambda w: w * 16384, 16384, 1, KT)]
    assert hit == [KT for KT in TILES if (KT - 1) % 3 != 2]
