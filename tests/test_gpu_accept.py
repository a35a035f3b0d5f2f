"""argus_accept_tokens on the GPU against the oracle's moves: rows are moved bit for bit, all else stays."""

import numpy as np
import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus
from mixed_precision_paged_argus_gb300 import workloads as W
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"


def case(Hkv, D, P, dtype, lens, new, paths, seed=0, width=None):
    rng = np.random.default_rng(seed)
    B = len(lens)
    s = dict(g=argus.geom(2 * Hkv, Hkv, D, P), P=P, lens=np.array(lens, np.int32), kind=dtype)
    s["q_start"] = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s["max_pages"] = max(1, max((n + P - 1) // P for n in lens))
    s["n_slots"] = B * s["max_pages"] + 2
    s["table"] = rng.permutation(s["n_slots"])[:B * s["max_pages"]].reshape(B, -1).astype(np.int32)
    s["codec"] = np.full(s["table"].shape, dtype, np.uint8)
    s["path"] = np.full((B, max([1] + [len(p) for p in paths]) if width is None else width), -7, np.int32)
    for b, p in enumerate(paths):
        s["path"][b, :len(p)] = p
    s["n_path"] = np.array([len(p) for p in paths], np.int32)
    s["pool"] = W.normal((s["n_slots"], 2, Hkv, P, D), dtype, seed + 1).to(DEV)
    return s


def run(s, status=None, stream=None):
    dev = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    out = torch.full((len(s["lens"]),), -9, dtype=torch.int32, device=DEV)
    argus.accept_tokens(s["g"], argus.Pool(s["kind"], s["pool"], None, s["n_slots"]), dev(s["codec"]), dev(s["table"]), s["max_pages"],
                        dev(s["q_start"]), dev(s["lens"]), dev(s["path"]), dev(s["n_path"]), out, status=status, stream=stream)
    torch.cuda.synchronize()
    return out.cpu().numpy()


def check(s):
    before = s["pool"].clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = run(s, status)
    moves, want, bad = oracle.accept_tokens(s["q_start"], s["lens"], s["path"], s["n_path"], s["P"], s["codec"], s["table"], s["kind"], s["n_slots"])
    ref = before.clone()
    for (a, ar), (z, zr) in moves:
        ref[z, :, :, zr] = before[a, :, :, ar]
    assert np.array_equal(lens, want) and int(status) == bad
    assert torch.equal(ref.view(torch.int16), s["pool"].view(torch.int16))
    return bad


@pytest.mark.parametrize("dtype", [W.FP16, W.BF16])
@pytest.mark.parametrize("Hkv,D,P", [(1, 64, 16), (2, 128, 16), (3, 64, 48), (8, 128, 64), (40, 128, 16)])
def test_paths(Hkv, D, P, dtype):
    paths = [[0, 2, 3, 9], [], [0, 1, 2], [25], list(range(26)), [3, 5, 7, 11, 13, 17, 19, 23, 24, 25]]
    s = case(Hkv, D, P, dtype, [26, 30, 100, 160, 57, 90], [26] * 6, paths, seed=Hkv + D)
    assert check(s) == 0


@pytest.mark.parametrize("seed", range(6))
def test_random_paths_longer_than_a_step(seed):
    """Paths of more than 32 tokens, which are looked up 32 at a time."""
    rng = np.random.default_rng(seed)
    B = int(rng.integers(1, 40))
    new = [int(rng.integers(0, 200)) for _ in range(B)]
    lens = [n + int(rng.integers(0, 300)) for n in new]
    paths = [sorted(rng.choice(n, size=int(rng.integers(0, n + 1)), replace=False).tolist()) if n else [] for n in new]
    assert check(case(2, 64, 16, W.FP16, lens, new, paths, seed=seed)) == 0


def test_what_is_not_a_path_is_cut_and_counted():
    paths = [[0, 3, 3, 5], [0, 2, 1], [-1, 2], [0, 26], [4, 5, 2 ** 31 - 1], [1, 2], list(range(1, 40))]
    s = case(2, 64, 16, W.FP16, [60] * 7, [26, 26, 26, 26, 26, 26, 39], paths, width=40)
    s["path"][6, 35] = 3                                 # behind the first 32
    s["n_path"][5] = -4
    assert check(s) == 7
    s["n_path"][:] = 1000                                # more than there are columns
    assert check(s) >= 7
    s["lens"][0] = 20                                    # shorter than its own tokens
    check(s)


def test_tokens_without_a_place_stay():
    s = case(2, 64, 16, W.FP16, [60, 60, 60], [30, 30, 30], [[1, 5, 20], [2, 3, 28], [0, 4]])
    s["table"][0, 1], s["codec"][1, 3], s["table"][2, 2] = -1, W.FP8_E4M3, s["n_slots"]
    s["lens"][2] = 500                                   # beyond the table
    assert check(s) > 0


def test_offsets_beyond_four_gigabytes_and_a_graph():
    s = case(8, 128, 16, W.BF16, [40, 77], [20, 30], [[0, 5, 19], [3, 28]], seed=3)
    n = (5 << 30) // (2 * 8 * 16 * 128 * 2)
    pool = torch.empty((n,) + tuple(s["pool"].shape[1:]), dtype=torch.bfloat16, device=DEV)
    pool[-s["n_slots"]:] = s["pool"]
    ref = {k: v for k, v in s.items()}
    ref["pool"] = s["pool"].clone()
    run(ref)
    s["table"] = s["table"] + (n - s["n_slots"]).__int__()
    s["table"], small, s["n_slots"] = s["table"].astype(np.int32), s["n_slots"], n
    start = pool[-small:].clone()
    s["pool"] = pool
    dev = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    t = [dev(s[k]) for k in ("codec", "table", "q_start", "lens", "path", "n_path")]
    out = torch.empty(2, dtype=torch.int32, device=DEV)
    g, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        argus.accept_tokens(s["g"], argus.Pool(s["kind"], pool, None, n), t[0], t[1], s["max_pages"], t[2], t[3], t[4], t[5], out)
    for _ in range(2):
        pool[-small:] = start
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool[-small:], ref["pool"]) and out.tolist() == [23, 49]
