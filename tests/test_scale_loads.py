"""The block-scaled kernel's waits count its loads of scales, which therefore have to
be vector loads, also where all lanes read one address (csrc/gated_common.hpp,
per_lane).  Compiled here, without a GPU: the same load with and without it."""
import os
import shutil
import subprocess

import pytest

from tiled_layout_algebra_amd import build as b

KERNEL = '''
#include "gated_common.hpp"
using namespace tla;
__global__ void probe(const GroupedParams p, float* out, int64_t at) {
  const float* s = p.sb + %s;
  float sum = 0.f;
  for (int k = 0; k < p.K; ++k) sum += s[(int64_t)k * p.sb_kb];
  out[threadIdx.x] = sum;
}
'''


def loads(expr, d):
    (d / "a.hip").write_text(KERNEL % expr)
    subprocess.run([b.HIPCC, *b.FLAGS, "-x", "hip", "--cuda-device-only", "-S", str(d / "a.hip"), "-o",
                    str(d / "a.s")], check=True, capture_output=True)
    text = (d / "a.s").read_text()
    loop = text[text.index("probe"):text.index("s_endpgm")]
    return sum("global_load_dword " in x for x in loop.splitlines()), "flat_load" in loop


@pytest.mark.skipif(not (os.path.exists(b.HIPCC) or shutil.which(b.HIPCC)), reason="needs hipcc")
def test_a_shared_address_is_loaded_by_vector_loads(tmp_path):
    assert loads("at", tmp_path)[0] == 0  # as the compiler likes it: scalar loads
    vector, flat = loads("per_lane(at)", tmp_path)
    assert vector > 0 and not flat
