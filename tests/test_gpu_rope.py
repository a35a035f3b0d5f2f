"""argus_rope_append on the GPU against the oracle's rotation.

Bound per element: the angle is exact to about 2^-40 of a turn, its sine and cosine to 2^-22
(fp32 fraction and sincospi), the two products and their sum to 3 * 2^-24 of
|x| + |y|; then half a step of the 16-bit type.
"""

import numpy as np
import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus
from mixed_precision_paged_argus_gb300 import workloads as W
import oracle
from oracle import codecs as C

pytestmark = pytest.mark.gpu
DEV = "cuda"


def to64(x):
    return (C.f16_bits_to_f64 if x.dtype == torch.float16 else C.bf16_bits_to_f64)(W.to_bits(x))


def case(Hq, Hkv, D, P, dtype, cached, new, rot, n_axes, seed, far=0, pair_axis="split"):
    rng = np.random.default_rng(seed)
    total, B = sum(new), len(new)
    lens = [a + n for a, n in zip(cached, new)]
    max_pages = max(1, max((n + P - 1) // P for n in lens))
    n_slots = B * max_pages + 3
    s = dict(g=argus.geom(Hq, Hkv, D, P), P=P, kind=dtype, lens=lens, max_pages=max_pages, n_slots=n_slots)
    s["table"] = rng.permutation(n_slots)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
    s["codec"] = np.full((B, max_pages), dtype, np.uint8)
    s["q_start"] = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s["qkv"] = W.normal((total, Hq + 2 * Hkv, D), dtype, seed).to(DEV)
    s["q"], s["k"], s["v"] = s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv], s["qkv"][:, Hq + Hkv:]
    s["pos"] = (far + rng.integers(0, 5000, (n_axes, total))).astype(np.int32)
    s["inv"] = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    s["axis"] = None if pair_axis is None else (np.arange(rot // 2) * n_axes // (rot // 2)).astype(np.uint8)
    s["pool"] = W.normal((n_slots, 2, Hkv, P, D), dtype, seed + 1).to(DEV)
    return s


def call(s, adjacent, q_out=None, status=None, stream=None):
    q_out = torch.full(s["q"].shape, float("nan"), dtype=s["q"].dtype, device=DEV) if q_out is None else q_out
    dev = lambda x: None if x is None else torch.from_numpy(x).to(DEV)  # noqa: E731
    argus.rope_append(s["g"], s["q"], s["k"], s["v"], q_out, dev(s["q_start"]), torch.tensor(s["lens"], dtype=torch.int32, device=DEV),
                      dev(s["pos"]), dev(s["inv"]), argus.Pool(s["kind"], s["pool"], None, s["n_slots"]), dev(s["codec"]),
                      dev(s["table"]), s["max_pages"], pair_axis=dev(s["axis"]), adjacent=adjacent, status=status, stream=stream)
    torch.cuda.synchronize()
    return q_out


def close(got, x64, ref, dtype):
    u = torch.finfo(dtype).eps / 2
    big = np.abs(x64).max(axis=-1, keepdims=True)       # |x| + |y| <= 2 max
    bound = u * np.abs(ref) + 2 * big * (2.0 ** -22 + 3 * 2.0 ** -24) * (1 + u) + torch.finfo(dtype).smallest_normal * u
    err = np.abs(got - ref)
    assert not np.isnan(got).any() and np.all(err <= bound), (err - bound).max()


def check(s, q_out, before, adjacent):
    dt = s["q"].dtype
    q64, k64 = to64(s["q"].contiguous()), to64(s["k"].contiguous())
    close(to64(q_out.contiguous()), q64, oracle.rotate(q64, s["pos"], s["inv"], s["axis"], adjacent), dt)
    kr = oracle.rotate(k64, s["pos"], s["inv"], s["axis"], adjacent)
    places = oracle.append_places(s["q_start"], s["lens"], s["P"], s["codec"], s["table"], s["kind"], s["n_slots"])
    after = s["pool"]
    left = before.clone()
    skipped = 0
    for t, at in places.items():
        if at is None:
            skipped += 1
            continue
        slot, row = at
        close(to64(after[slot, 0, :, row].contiguous()), k64[t], kr[t], dt)
        assert torch.equal(after[slot, 1, :, row], s["v"][t])
        left[slot, :, :, row] = after[slot, :, :, row]
    assert torch.equal(left, after)                     # every other row as it was
    return skipped


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 16), (64, 64), (128, 32), (128, 96), (128, 128)])
@pytest.mark.parametrize("dtype,n_axes", [(W.FP16, 1), (W.BF16, 3), (W.FP16, 4), (W.BF16, 2)])
def test_rotation_and_append(dtype, n_axes, D, rot, adjacent):
    s = case(6, 2, D, 16, dtype, [0, 15, 100], [17, 1, 40], rot, n_axes, seed=D + rot + n_axes)
    before = s["pool"].clone()
    assert check(s, call(s, adjacent), before, adjacent) == 0


@pytest.mark.parametrize("far", [10 ** 6, 2 ** 31 - 5001, -2 ** 31])
def test_far_and_negative_positions(far):
    s = case(2, 1, 64, 16, W.FP16, [0], [33], 64, 1, seed=7, far=far, pair_axis=None)
    before = s["pool"].clone()
    check(s, call(s, False), before, False)


def test_position_zero_is_the_identity():
    s = case(4, 2, 128, 16, W.BF16, [5], [3], 128, 3, seed=8)
    s["pos"][:] = 0
    assert torch.equal(call(s, True), s["q"])


@pytest.mark.parametrize("batch", [1, 33, 300, 900])
def test_many_sequences_and_empty_ones(batch):
    rng = np.random.default_rng(batch)
    new = rng.integers(0, 3, batch).tolist()
    new[-1] = 1
    s = case(2, 1, 64, 16, W.FP16, rng.integers(0, 40, batch).tolist(), new, 32, 2, seed=batch)
    before = s["pool"].clone()
    assert check(s, call(s, False), before, False) == 0


def test_in_place_queries():
    s = case(4, 2, 128, 16, W.BF16, [3], [20], 64, 2, seed=9)
    ref = call(s, False)
    qkv = s["qkv"].clone()
    s["q"] = qkv[:, :4]
    assert torch.equal(call(s, False, q_out=s["q"]), ref) and torch.equal(qkv[:, 4:], s["qkv"][:, 4:])


def test_tokens_without_a_place_and_unknown_axes_are_counted():
    s = case(2, 1, 64, 16, W.FP16, [0, 30, 0], [20, 10, 5], 32, 2, seed=10)
    s["table"][0, 1], s["table"][1, 2] = -1, s["n_slots"]
    s["codec"][2, 0] = W.FP8_E4M3
    before = s["pool"].clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    skipped = check(s, call(s, False, status=status), before, False)
    assert skipped == 4 + 8 + 5 and int(status) == skipped
    s["axis"][3] = 2
    status.zero_()
    before = s["pool"].clone()
    check(s, call(s, False, status=status), before, False)
    assert int(status) == skipped + 35
    # lengths shorter than the new tokens: the first ones have no place
    s = case(2, 1, 64, 16, W.FP16, [0], [20], 32, 2, seed=12)
    s["lens"] = [12]
    before = s["pool"].clone()
    assert check(s, call(s, True), before, True) == 8


def test_rows_of_no_sequence_are_left():
    s = case(2, 1, 64, 16, W.FP16, [0], [9], 32, 1, seed=13)
    s["q_start"] = np.array([2, 7], np.int32)
    s["lens"] = [5]
    before = s["pool"].clone()
    out = call(s, False)
    assert torch.isnan(out[:2]).all() and torch.isnan(out[7:]).all() and not torch.isnan(out[2:7]).any()
    assert int((before != s["pool"]).any(-1).any(1).any(1).sum()) == 5


def test_replayed_from_a_graph_on_another_stream():
    s = case(6, 2, 128, 16, W.BF16, [5, 100], [3, 40], 96, 3, seed=20)
    ref = call(s, False)
    stored = s["pool"].clone()
    dev = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    tensors = [dev(s["q_start"]), torch.tensor(s["lens"], dtype=torch.int32, device=DEV), dev(s["pos"]), dev(s["inv"])]
    codec, table, axis = dev(s["codec"]), dev(s["table"]), dev(s["axis"])
    q_out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=DEV)
    pool = argus.Pool(s["kind"], s["pool"], None, s["n_slots"])
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        argus.rope_append(s["g"], s["q"], s["k"], s["v"], q_out, tensors[0], tensors[1], tensors[2], tensors[3], pool, codec, table,
                          s["max_pages"], pair_axis=axis)
    for _ in range(2):
        q_out.zero_()
        s["pool"].copy_(stored * 0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q_out, ref)
    places = oracle.append_places(s["q_start"], s["lens"], s["P"], s["codec"], s["table"], s["kind"], s["n_slots"])
    for slot, row in places.values():
        assert torch.equal(s["pool"][slot, :, :, row], stored[slot, :, :, row])


def test_large_ragged_batches():
    """Thousands of tokens, so that warps loop over tokens; sequences of very different lengths."""
    rng = np.random.default_rng(21)
    new = [4000, 1, 0, 700, 33] + rng.integers(0, 60, 60).tolist()
    s = case(2, 1, 64, 16, W.FP16, rng.integers(0, 900, len(new)).tolist(), new, 64, 3, seed=22)
    before = s["pool"].clone()
    assert check(s, call(s, True), before, True) == 0
