"""argus_norm_rope_append at the largest eps that its documentation allows, where the mean square's sum with it leaves fp32."""

import pytest

from mixed_precision_paged_argus_gb300 import workloads as W
from test_gpu_norm_rope import call, check, weights
from test_gpu_rope import case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [1e-3, 1e15, 1e18, 3e18, 1e19, 1e30])
@pytest.mark.parametrize("eps", [float.fromhex("0x1.fffffep+127"), 3e38])
def test_largest_eps(scale, eps):
    s = case(4, 2, 128, 16, W.BF16, [5], [9], 128, 1, seed=4)
    s["qkv"].mul_(scale)
    w, before = weights(128, 1) * 16, s["pool"].clone()
    check(s, w.astype("float32"), call(s, w.astype("float32"), eps=eps), before, eps=eps)
