"""argus_rope_append: the angle's fraction of a turn at far positions and high frequencies.

The fraction is 64-bit fixed point, off by at most 2^-64 per position (the rounding of the frequency's fraction, and of
the fraction of a product of two doubles with 106 bits), so by at most 2^-33 of a turn at position 2^31: below
the 2^-25 of its fp32 form.  Bounds as in test_gpu_rope.
"""

import numpy as np
import pytest

from mixed_precision_paged_argus_gb300 import workloads as W
from test_gpu_rope import call, case, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("far", [0, 10 ** 6, 2 ** 31 - 5001, -2 ** 31])
@pytest.mark.parametrize("top", [100.0, 1e6, 1e12])
def test_high_frequencies(top, far, adjacent):
    s = case(2, 1, 128, 16, W.FP16, [0], [33], 128, 2, seed=30, far=far)
    s["inv"] = top ** np.linspace(-1, 1, 64) * (1 + 1e-3 * np.random.default_rng(31).standard_normal(64))
    before = s["pool"].clone()
    check(s, call(s, adjacent), before, adjacent)


def test_frequencies_at_whole_turns():
    """Frequencies next to multiples of a turn, whose fractions are next to 0 and 1, and frequency 0."""
    s = case(2, 1, 64, 16, W.FP16, [0], [33], 64, 1, seed=32, far=2 ** 31 - 5001)
    turns = np.concatenate([np.arange(1, 9), 2.0 ** np.arange(8), 10.0 ** np.arange(8)]) * (2 * np.pi)
    s["inv"] = np.concatenate([turns, np.nextafter(turns[:7], 0), [0.0]])
    before = s["pool"].clone()
    check(s, call(s, False), before, False)
