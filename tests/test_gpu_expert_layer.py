"""The expert layer end to end: forward, backward and int8 decoding against
float64.  Bounds: a bf16 output is off by at most half a step, 2^-9 of its
value; what enters a product rounded that way (the activation, z, dz) moves the
product by a like share of its terms' magnitudes, which the sums' largest value
exceeds the root mean square of by far less than 8, so 8 2^-9 of the largest
value covers each chain of two rounded factors.  int8 rounds x, the activation
and both weights to 1/254 of each row's largest value (about 4 standard
deviations), so a term is off by at most 4/254 of its factors' spread, on each
side of each product: at most 4 * 4/254 of the largest value."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [3, 1000])
def test_layer_against_float64(rows):
    from tiled_layout_algebra_amd.expert_layer import example
    for name, err in example(rows).items():
        assert err <= (16 / 254 if "int8" in name else 8 * 2.0 ** -9), (name, err)
