"""All frequencies and gains of the library's rotary plans against the oracle's own definition of them."""
import numpy as np
import pytest

import exact_top_token_amd as hk
from oracle import operators as op

# dim, base, factor, original: usual models' ranges, ramps cut off at both ends, a ramp between neighbouring pairs, contexts below a turn
PLANS = [
    (64, 10000.0, 4.0, 4096), (64, 10000.0, 40.0, 4096), (128, 1000000.0, 4.0, 32768), (64, 1000000.0, 32.0, 32768), (128, 500000.0, 8.0, 8192),
    (32, 10000.0, 2.5, 131072), (64, 10000.0, 4.0, 1 << 31), (64, 100.0, 3.0, 100000), (64, 10000.0, 16.0, 100), (64, 10000.0, 16.0, 7),
    (64, 10000.0, 8.0, 6), (64, 10000.0, 8.0, 1), (2, 10000.0, 8.0, 4096), (4, 10000.0, 8.0, 4096), (6, 1.5, 8.0, 300), (1024, 10000.0, 1.0, 4096),
    (600, 1e9, 1e6, 1 << 20), (64, 1.0001, 4.0, 4096), (16, 1e30, 4.0, 64),
]


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("plan", PLANS)
def test_frequencies_and_gain(plan, scaling):
    dim, base, factor, original = plan
    got = hk.Rotary(dim, base=base, scaling=scaling, factor=factor, original=original, device="cpu")
    f, gain = op.rotary_plan(dim, base, scaling, factor, original)
    assert got.freq.shape == (dim // 2,)
    # powers of 64-bit arguments up to 70 in base 2, a few roundings more
    assert np.allclose(got.freq.numpy(), f, rtol=1e-13, atol=0), np.argmax(np.abs(got.freq.numpy() / f - 1))
    assert abs(got.gain - gain) <= 4e-16 * gain


def test_the_ramp_by_hand():
    """dim 8, base 10^4: pairs at 1, 0.1, 0.01, 0.001 radians.  In 20,000 positions they make 3183, 318, 31.8 and 3.18 turns;
    the number at which 32 turns fall is 1.998, at which one falls 3.503: the ramp runs from 1 to 4."""
    f = hk.Rotary(8, scaling="yarn", factor=5.0, original=20000, device="cpu").freq.numpy()
    want = [1.0, 0.1, 0.01 * (2 / 3 + 1 / 3 / 5), 0.001 * (1 / 3 + 2 / 3 / 5)]
    assert np.allclose(f, want, rtol=1e-13, atol=0)
