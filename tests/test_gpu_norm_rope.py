"""argus_norm_rope_append on the GPU against the oracle's norms and rotation.

Bound per element: the sum of D squares in fp32 is off by at most D 2^-24 of itself, the root of its mean by half of
that, 1 / sqrt by 2^-22, three products by 2^-24 each; then the rotation's bound (test_gpu_rope.py) on the normed
values, and half a step of the 16-bit type.
"""

import numpy as np
import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus
from mixed_precision_paged_argus_gb300 import workloads as W
import oracle
from test_gpu_rope import DEV, case, to64

pytestmark = pytest.mark.gpu
EPS = 1e-6


def weights(d, seed):
    return (1.0 + 0.3 * np.random.default_rng(seed).standard_normal((2, d))).astype(np.float32)


def call(s, w, adjacent=False, eps=EPS, q_out=None, status=None):
    q_out = torch.full(s["q"].shape, float("nan"), dtype=s["q"].dtype, device=DEV) if q_out is None else q_out
    dev = lambda x: None if x is None else torch.from_numpy(x).to(DEV)  # noqa: E731
    argus.norm_rope_append(s["g"], s["q"], s["k"], s["v"], q_out, dev(s["q_start"]), torch.tensor(s["lens"], dtype=torch.int32, device=DEV),
                           dev(s["pos"]), dev(s["inv"]), argus.Pool(s["kind"], s["pool"], None, s["n_slots"]), dev(s["codec"]), dev(s["table"]),
                           s["max_pages"], dev(w[0]), dev(w[1]), eps, pair_axis=dev(s["axis"]), adjacent=adjacent, status=status)
    torch.cuda.synchronize()
    return q_out


def close(got, x, w, s, adjacent, dtype, eps):
    y = oracle.head_norm(x, w, eps)
    ref = oracle.rotate(y, s["pos"], s["inv"], s["axis"], adjacent)
    u, d = torch.finfo(dtype).eps / 2, x.shape[-1]
    rel = d * 2.0 ** -25 + 2.0 ** -22 + 3 * 2.0 ** -24
    big = np.abs(y).max(-1, keepdims=True)
    bound = u * np.abs(ref) + 2 * big * (rel + 2.0 ** -22 + 3 * 2.0 ** -24) * (1 + u) + torch.finfo(dtype).smallest_normal * u
    err = np.abs(got - ref)
    assert not np.isnan(got).any() and np.all(err <= bound), (err - bound).max()


def check(s, w, q_out, before, adjacent=False, eps=EPS):
    dt = s["q"].dtype
    q64, k64 = to64(s["q"].contiguous()), to64(s["k"].contiguous())
    close(to64(q_out.contiguous()), q64, w[0], s, adjacent, dt, eps)
    places = oracle.append_places(s["q_start"], s["lens"], s["P"], s["codec"], s["table"], s["kind"], s["n_slots"])
    stored = np.zeros(k64.shape)
    left = before.clone()
    kept = [t for t, at in places.items() if at is not None]
    for t in kept:
        slot, row = places[t]
        stored[t] = to64(s["pool"][slot, 0, :, row].contiguous())
        assert torch.equal(s["pool"][slot, 1, :, row], s["v"][t])
        left[slot, :, :, row] = s["pool"][slot, :, :, row]
    y = oracle.rotate(oracle.head_norm(k64, w[1], eps), s["pos"], s["inv"], s["axis"], adjacent)
    stored[[t for t in range(len(stored)) if t not in set(kept)]] = y[[t for t in range(len(stored)) if t not in set(kept)]]
    close(stored, k64, w[1], s, adjacent, dt, eps)
    assert torch.equal(left, s["pool"])                 # every other row as it was


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 16), (64, 64), (128, 32), (128, 96), (128, 128)])
@pytest.mark.parametrize("dtype,Hq,Hkv", [(W.FP16, 6, 2), (W.BF16, 14, 2), (W.FP16, 1, 1), (W.BF16, 32, 8)])
def test_norms_rotation_and_append(dtype, Hq, Hkv, D, rot, adjacent):
    s = case(Hq, Hkv, D, 16, dtype, [0, 15, 100], [17, 1, 40], rot, 2, seed=D + rot + Hq)
    w, before = weights(D, rot), s["pool"].clone()
    check(s, w, call(s, w, adjacent), before, adjacent)


@pytest.mark.parametrize("which", [0, 1])
def test_without_weights(which):
    s = case(4, 2, 128, 16, W.BF16, [5], [9], 128, 1, seed=4)
    w, before = list(weights(128, 1)), s["pool"].clone()
    w[which] = None
    check(s, w, call(s, w), before)


@pytest.mark.parametrize("scale,eps", [(1e30, 1e-6), (3e38, 1e-6), (1e-20, 1e-6), (1e-12, 1e-20), (1.0, 1e4), (0.0, 1e-6)])
def test_magnitudes_at_the_ends(scale, eps):
    """bf16 reaches as far as fp32: squares beyond it, and squares far below eps."""
    s = case(4, 2, 64, 16, W.BF16, [0], [21], 32, 1, seed=5)
    big = (s["qkv"].float() / s["qkv"].float().abs().max()) * scale
    s["qkv"].copy_(big.to(torch.bfloat16))
    w, before = weights(64, 2), s["pool"].clone()
    check(s, w, call(s, w, eps=eps), before, eps=eps)


def test_fp16s_largest_values():
    s = case(4, 2, 128, 16, W.FP16, [0], [21], 32, 1, seed=6)
    s["qkv"].copy_((s["qkv"].float() / s["qkv"].float().abs().max() * 65504).half())
    w, before = weights(128, 2), s["pool"].clone()
    check(s, w, call(s, w), before)


def test_infinities_and_nans_stay_in_their_heads():
    s = case(8, 2, 128, 16, W.BF16, [3], [12], 64, 1, seed=7)
    w = weights(128, 3)
    clean = call(s, w).clone()
    pool = s["pool"].clone()
    s["q"][3, 5, 100], s["q"][4, 0, 7], s["k"][2, 1, 9] = float("nan"), float("inf"), float("nan")
    got = call(s, w)
    hit = torch.zeros((12, 8), dtype=torch.bool, device=DEV)
    hit[3, 5] = hit[4, 0] = True
    assert torch.isnan(got[3, 5]).all() and torch.isnan(got[4, 0, 7]) and torch.equal(got[~hit], clean[~hit])
    places = oracle.append_places(s["q_start"], s["lens"], 16, s["codec"], s["table"], s["kind"], s["n_slots"])
    slot, row = places[2]
    assert torch.isnan(s["pool"][slot, 0, 1, row]).all()
    s["pool"][slot, 0, 1, row] = pool[slot, 0, 1, row]
    assert torch.equal(s["pool"], pool)


@pytest.mark.parametrize("new", [[1] * 40, [700, 0, 2500, 3], [1]])
def test_batch_shapes(new):
    """Few tokens take several warps each, many share them."""
    s = case(14, 2, 64, 1024, W.FP16, list(range(len(new))), new, 64, 3, seed=len(new))
    w, before = weights(64, 4), s["pool"].clone()
    check(s, w, call(s, w), before)


def test_in_place_skipped_tokens_and_other_rows():
    s = case(4, 2, 128, 16, W.BF16, [3, 30], [20, 10], 64, 2, seed=9)
    w = weights(128, 5)
    ref = call(s, w)
    qkv = s["qkv"].clone()
    s["q"] = qkv[:, :4]
    assert torch.equal(call(s, w, q_out=s["q"]), ref) and torch.equal(qkv[:, 4:], s["qkv"][:, 4:])
    s = case(2, 1, 64, 16, W.FP16, [0, 30, 0], [20, 10, 5], 32, 2, seed=10)
    s["table"][0, 1], s["codec"][2, 0] = -1, W.FP8_E4M3
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    before, w = s["pool"].clone(), weights(64, 6)
    check(s, w, call(s, w, status=status), before)
    assert int(status) == 4 + 5


def test_replayed_from_a_graph():
    s = case(6, 2, 128, 16, W.BF16, [5, 100], [3, 40], 96, 3, seed=20)
    w = weights(128, 7)
    ref = call(s, w)
    dev = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    t = [dev(s["q_start"]), torch.tensor(s["lens"], dtype=torch.int32, device=DEV), dev(s["pos"]), dev(s["inv"])]
    codec, table, axis, wq, wk = dev(s["codec"]), dev(s["table"]), dev(s["axis"]), dev(w[0]), dev(w[1])
    q_out = torch.empty_like(ref)
    pool = argus.Pool(s["kind"], s["pool"], None, s["n_slots"])
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        argus.norm_rope_append(s["g"], s["q"], s["k"], s["v"], q_out, t[0], t[1], t[2], t[3], pool, codec, table, s["max_pages"], wq, wk, EPS,
                               pair_axis=axis)
    q_out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out, ref)
