"""argus_fork_pages after rows were shortened: their pages behind the new end given back by the caller, as the header says."""

import numpy as np
import pytest

from mixed_precision_paged_argus_gb300 import workloads as W
import oracle
from test_gpu_pages import check_fork, table_case

pytestmark = pytest.mark.gpu


def shorten(s, lens):
    for b, n in enumerate(lens):
        for j in range((n + s["P"] - 1) // s["P"], (s["lens"][b] + s["P"] - 1) // s["P"]):
            s["refs"][s["codec"][b, j]][s["table"][b, j]] -= 1
            s["table"][b, j], s["codec"][b, j] = -1, 0
    s["lens"] = np.minimum(s["lens"], np.array(lens, np.int32))


def test_a_rejected_page_is_free_again():
    s = table_case(1, 16, 6, [40], {W.FP16: 9}, 1, shared=0, held=0)
    s["refs"][W.FP16][:] = 0
    s["table"][0, :3] = [5, 6, 7]
    s["refs"][W.FP16][5:8] = 1
    shorten(s, [30])
    check_fork(s, [0], [20], W.FP16)
    t, _, n, refs, _, st = oracle.fork_pages([0], [20], W.FP16, s["slots"], s["refs"], s["codec"], s["table"], s["lens"], 16)
    assert t[0].tolist() == [5, 6, 0, 1, -1, -1] and n.tolist() == [50] and st == 0
    assert refs[W.FP16].tolist() == [1, 1, 0, 0, 0, 1, 1, 0, 0]


@pytest.mark.parametrize("seed", range(4))
def test_counts_stay_the_references(seed):
    rng = np.random.default_rng(seed)
    B, P, max_pages = 20, 16, 16
    s = table_case(B, P, max_pages, rng.integers(0, 12 * P, B).tolist(), {W.BF16: 400, W.INT8: 400}, seed, held=0)
    for _ in range(4):
        shorten(s, [int(max(0, n - rng.integers(0, 40))) for n in s["lens"]])
        parents = [int(rng.integers(-1, B)) if rng.random() < 0.4 else b for b in range(B)]
        new = rng.integers(0, 20, B).tolist()
        check_fork(s, parents, new, W.BF16)
        t, c, n, refs, _, st = oracle.fork_pages(parents, new, W.BF16, s["slots"], s["refs"], s["codec"], s["table"], s["lens"], P)
        assert st == 0
        s["table"], s["codec"], s["lens"], s["refs"] = t, c, n.astype(np.int32), {k: v.astype(np.int32) for k, v in refs.items()}
        for k in s["slots"]:
            held = np.zeros(s["slots"][k], int)
            for b in range(B):
                for j in range((s["lens"][b] + P - 1) // P):
                    if c[b, j] == k:
                        held[t[b, j]] += 1
            assert np.array_equal(held, refs[k])
