"""argus_paged_extend_attn with V scales anywhere in the fp32 range: the sum of the weights knows nothing of them.

Bounds as in test_gpu_extend, u = eps / 2 of the 16-bit type, e the score's and 2^x's error:
  |o - ref| <= u sum p|v| + u |ref| + 2 e sum p|v| + 2^-32 max_j (p_j s_j) sum_j |code_j| / sum p,
plus, where scales beyond 2^64 move the sum's reference by 32: one fp32 difference near 32 (half a step of
2^-18) in the exponent and one log2 near -32 (half a step of 2^-18), together below 2^-18 of a bit,
hence 2^-18 in lse2 and 2^-18 sum p|v| in o.
"""

import math

import numpy as np
import pytest
import torch

from mixed_precision_paged_argus_gb300 import workloads as W
import oracle
from test_gpu_extend import F8, I8, make, run

pytestmark = pytest.mark.gpu


def rescale(c, exponents, k_factor, seed):
    """V scales times 2^x, x drawn from the exponents; K scales times k_factor."""
    rng = np.random.default_rng(seed)
    for pool in c.pools:
        codes, meta = c.opools[pool.codec]
        if meta is not None:
            meta[:, 1] = (meta[:, 1] * 2.0 ** rng.choice(exponents, size=meta[:, 1].shape)).astype(np.float32)
            meta[:, 0] *= np.float32(k_factor)
            pool.meta.copy_(torch.from_numpy(meta))


def check(c, out, lse, causal):
    q64 = c.to64(W.to_bits(c.q))
    ref, ref_lse, bad, av, pc, qk, smax = oracle.paged_extend(q64, c.q_start, c.Hkv, c.P, c.opools, c.page_codec, c.table, c.lens,
                                                          c.scale, causal)
    assert bad == 0
    fi = torch.finfo(out.dtype)
    u = fi.eps / 2
    e = (math.log(2) * (c.D * 2.0 ** -23 * qk + 2.0 ** -22 * smax) + 2.0 ** -21)[..., None]
    lb = c.D * 2.0 ** -23 * qk + 2.0 ** -22 * smax + 2.0 ** -19 + 2.0 ** -18 + 2.0 ** -22 * np.abs(ref_lse)
    gl = lse.cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(gl)) and np.all(np.abs(gl - ref_lse) <= lb), (np.abs(gl - ref_lse) - lb).max()
    got = out.float().cpu().numpy().astype(np.float64)
    bound = u * av + u * np.abs(ref) + (2 * e + 2.0 ** -18) * av + 2.0 ** -32 * pc + fi.smallest_normal * fi.eps
    over = np.abs(got - ref) / bound
    assert not np.isnan(got).any() and over.max() <= 1, over.max()


# what a page's V scale (some 2^-7 at first) is multiplied by
RANGES = {"sixty": [-60, 60], "thirty": [-34, -20, 0, 20, 34], "far up": [-20, 0, 20, 100, 110], "one far up": [-20] * 30 + [116],
          "far down": [-130, -110], "down and up": [-40, 70], "all": list(range(-130, 116))}


@pytest.mark.parametrize("n_q", [1, 12, 20])        # with four heads per KV head: 4, 48 and 80 rows, the three layouts of a tile
@pytest.mark.parametrize("codecs", [[F8, I8], [W.BF16, F8, I8]])
@pytest.mark.parametrize("name", list(RANGES))
def test_scales_far_apart(name, codecs, n_q):
    c = make(8, 2, 128, 16, [900, 300], [n_q, n_q], codecs, W.BF16, seed=700 + n_q)
    rescale(c, RANGES[name], 4.0, seed=len(name) + n_q)
    out, lse = run(c, True)
    check(c, out, lse, True)


@pytest.mark.parametrize("name", ["far up", "sixty", "all"])
def test_scales_far_apart_over_cut_items(name):
    """One sequence over all CTAs: pieces of very different scales are joined."""
    c = make(4, 1, 64, 16, [6000], [3], [F8], W.BF16, seed=750)
    rescale(c, RANGES[name], 4.0, seed=751)
    out, lse = run(c, False)
    check(c, out, lse, False)


def test_small_scales_with_fp16_queries():
    c = make(8, 2, 64, 16, [700, 40], [5, 33], [F8, I8], W.FP16, seed=760)
    rescale(c, list(range(-130, 1, 10)), 4.0, seed=761)
    out, lse = run(c, True)
    check(c, out, lse, True)


def test_a_far_scale_weighs_nothing():
    """Equal scores: lse2 is log2 of the number of positions whatever the scales are, and the mean counts every page."""
    c = make(2, 1, 64, 16, [320], [2], [I8], W.BF16, seed=770)
    rescale(c, [0], 0.0, seed=0)
    codes, meta = c.opools[I8]
    for far in (2.0 ** 40, 2.0 ** 100, 2.0 ** 120, 2.0 ** -60, 2.0 ** -140, 0.0):
        meta[:, 1] = 2.0 ** -24
        meta[c.table[0, 7], 1] = far
        c.pools[0].meta.copy_(torch.from_numpy(meta))
        out, lse = run(c, False)
        assert (lse - math.log2(320)).abs().max() <= 2.0 ** -17, far
        check(c, out, lse, False)
