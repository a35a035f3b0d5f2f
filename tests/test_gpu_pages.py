"""argus_fork_pages and argus_compact_pages on the GPU: equal to the oracle's table, counts and copies."""

import numpy as np
import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus
from mixed_precision_paged_argus_gb300 import workloads as W
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"
ALL = [W.FP16, W.BF16, W.FP8_E4M3, W.INT8, W.INT4_G32, W.INT2_G32, W.INT1_G32]


def fill(pool, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    for t in (pool.codes, pool.meta):
        if t is not None:
            b = t.view(torch.uint8)
            b.copy_(torch.randint(0, 256, b.shape, generator=g, device=DEV, dtype=torch.uint8))


def table_case(B, P, max_pages, lens, slots, seed, shared=0.3, held=0.2, Hkv=2, D=64):
    """slots: dict codec -> number.  Rows hold pages of random tiers; some are shared between rows or held outside."""
    rng = np.random.default_rng(seed)
    table = np.full((B, max_pages), -1, np.int32)
    codec = np.zeros((B, max_pages), np.uint8)
    refs = {c: np.zeros(n, np.int32) for c, n in slots.items()}
    free = {c: rng.permutation(n).tolist() for c, n in slots.items()}
    for b in range(B):
        for j in range((lens[b] + P - 1) // P):
            donors = [a for a in range(b) if lens[a] > j * P]
            if donors and rng.random() < shared:
                a = donors[rng.integers(len(donors))]
                codec[b, j], table[b, j] = codec[a, j], table[a, j]
            else:
                have = [c for c in slots if free[c]]
                c = have[rng.integers(len(have))]
                codec[b, j], table[b, j] = c, free[c].pop()
            refs[codec[b, j]][table[b, j]] += 1
    for c in slots:
        used = refs[c] > 0
        refs[c][used & (rng.random(slots[c]) < held)] += 1
    pools = []
    for c, n in slots.items():
        pools.append(argus.Pool.empty(c, n, Hkv, P, D, device=DEV))
        fill(pools[-1], seed + c)
    return dict(B=B, P=P, max_pages=max_pages, lens=np.array(lens, np.int32), table=table, codec=codec, refs=refs, pools=pools,
                slots=slots, g=argus.geom(Hkv, Hkv, D, P))


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def bytes_of(pool):
    return [None if t is None else t.view(torch.uint8).clone() for t in (pool.codes, pool.meta)]


def run_fork(s, parents, n_new, new_codec, stream=None):
    t = torch.full((s["B"], s["max_pages"]), 77, dtype=torch.int32, device=DEV)
    c = torch.full((s["B"], s["max_pages"]), 77, dtype=torch.uint8, device=DEV)
    n = torch.full((s["B"],), 77, dtype=torch.int32, device=DEV)
    rin = [dev(s["refs"][p.codec]) for p in s["pools"]]
    rout = [torch.full_like(r, 77) for r in rin]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.full((argus.fork_workspace_bytes(s["B"], s["pools"]),), 0xFF, dtype=torch.uint8, device=DEV)
    argus.fork_pages(s["g"], dev(np.array(parents, np.int32)), None if n_new is None else dev(np.array(n_new, np.int32)), new_codec,
                     s["pools"], rin, rout, dev(s["codec"]), dev(s["table"]), dev(s["lens"]), c, t, n, s["max_pages"], ws,
                     status=status, stream=stream)
    torch.cuda.synchronize()
    return t.cpu().numpy(), c.cpu().numpy(), n.cpu().numpy(), {p.codec: r.cpu().numpy() for p, r in zip(s["pools"], rout)}, int(status)


def check_fork(s, parents, n_new, new_codec):
    before = {p.codec: bytes_of(p) for p in s["pools"]}
    t, c, n, r, st = run_fork(s, parents, n_new, new_codec)
    ot, oc, on, orf, copies, ost = oracle.fork_pages(parents, n_new, new_codec, s["slots"], s["refs"], s["codec"], s["table"], s["lens"], s["P"])
    assert np.array_equal(t, ot) and np.array_equal(c, oc) and np.array_equal(n, on) and st == ost
    for k in s["slots"]:
        assert np.array_equal(r[k], orf[k]), k
    for p in s["pools"]:
        want = before[p.codec]
        for codec, src, dst in copies:
            if codec == p.codec:
                for x in want:
                    if x is not None:
                        x[dst] = x[src]
        for x, y in zip(want, bytes_of(p)):
            assert x is None or torch.equal(x, y)
    return copies, st


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("codecs", [[W.FP16], [W.BF16, W.FP8_E4M3], ALL])
def test_fork_matches_the_oracle(codecs, seed):
    rng = np.random.default_rng(seed)
    B, P, max_pages = int(rng.integers(1, 40)), 16, 24
    lens = rng.integers(0, 20 * P, B).tolist()
    s = table_case(B, P, max_pages, lens, {c: 900 for c in codecs}, seed)
    parents = [int(rng.integers(-1, B)) if rng.random() < 0.6 else b for b in range(B)]
    n_new = rng.integers(0, 40, B).tolist()
    check_fork(s, parents, n_new, codecs[0])


def test_fork_of_a_beam_shares_and_copies():
    """Eight beams of one parent: all get its pages; the first keeps the partial one only if nobody else holds it."""
    for held in (0.0, 1.0):
        s = table_case(8, 16, 10, [70] + [0] * 7, {W.FP16: 64}, 3, shared=0, held=held)
        copies, st = check_fork(s, [0] * 8, [1] * 8, W.FP16)
        assert len(copies) == (8 if held else 7) and st == 0
        s = table_case(8, 16, 10, [70] + [0] * 7, {W.FP16: 64}, 3, shared=0, held=held)
        assert check_fork(s, [0] * 8, None, W.FP16)[0] == []          # nobody writes: nothing is copied
        s = table_case(8, 16, 10, [64] + [0] * 7, {W.FP16: 64}, 3, shared=0, held=held)
        assert check_fork(s, [0] * 8, [1] * 8, W.FP16)[0] == []       # a full last page is never written


def test_fork_swaps_rows_and_frees():
    s = table_case(4, 32, 8, [100, 33, 256, 0], {W.BF16: 40, W.INT8: 40}, 5, shared=0.2)
    check_fork(s, [1, 0, -1, 2], [0, 64, 5, 0], W.BF16)


def test_freed_slots_are_used_at_once():
    s = table_case(2, 16, 4, [64, 16], {W.FP16: 5}, 6, shared=0, held=0)
    copies, st = check_fork(s, [-1, 1], [9, 48], W.FP16)
    assert st == 0


def test_fork_without_free_slots_and_with_anomalies_counts():
    s = table_case(3, 16, 4, [40, 20, 10], {W.FP16: 6}, 7, shared=0, held=0)
    copies, st = check_fork(s, [0, 0, 2], [24, 40, 40], W.FP16)
    assert st > 0
    s = table_case(4, 16, 4, [40, 20, 10, 64], {W.FP16: 40, W.FP8_E4M3: 40}, 8)
    s["table"][0, 1] = 1000
    s["table"][1, 1] = -3                   # a partial last page that names no slot
    s["lens"][3] = 90                       # beyond the table
    check_fork(s, [7, 1, -9, 0], [3, 3, 3, -2], W.FP16)
    check_fork(s, [0, 1, 2, 3], [100, 3, 3, 2], W.FP8_E4M3)


@pytest.mark.parametrize("P,Hkv,D", [(1024, 2, 64), (16, 8, 128), (48, 1, 64)])
def test_fork_large_batches_and_pools(P, Hkv, D):
    rng = np.random.default_rng(P)
    B, max_pages = 300, 12
    lens = rng.integers(0, 8 * P, B).tolist()
    n = {1024: 2500, 16: 9000, 48: 5000}[P]
    s = table_case(B, P, max_pages, lens, {W.FP16: n, W.INT4_G32: 2500}, P, Hkv=Hkv, D=D)
    parents = [int(rng.integers(-1, B)) if rng.random() < 0.4 else b for b in range(B)]
    check_fork(s, parents, rng.integers(0, 2 * P, B).tolist(), W.FP16)


def run_compact(s, pool):
    t = torch.full((s["B"], s["max_pages"]), 77, dtype=torch.int32, device=DEV)
    rin = dev(s["refs"][pool.codec])
    rout = torch.full_like(rin, 77)
    n_live = torch.full((1,), 77, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.full((argus.compact_workspace_bytes(pool),), 0xFF, dtype=torch.uint8, device=DEV)
    argus.compact_pages(s["g"], pool, rin, rout, dev(s["codec"]), dev(s["table"]), dev(s["lens"]), t, s["max_pages"], n_live, ws,
                        status=status)
    torch.cuda.synchronize()
    return t.cpu().numpy(), rout.cpu().numpy(), int(n_live), int(status)


def check_compact(s, pool):
    before = bytes_of(pool)
    t, r, n, st = run_compact(s, pool)
    ot, orf, moves, on, ost = oracle.compact_pages(pool.codec, s["refs"][pool.codec], s["codec"], s["table"], s["lens"], s["P"])
    assert np.array_equal(t, ot) and np.array_equal(r, orf) and (n, st) == (on, ost)
    for x in before:
        for src, dst in moves:
            if x is not None:
                x[dst] = x[src]
    for x, y in zip(before, bytes_of(pool)):
        assert x is None or torch.equal(x, y)
    return moves


@pytest.mark.parametrize("codec", ALL)
@pytest.mark.parametrize("n_slots", [1, 60, 1023, 1024, 1025, 5000])
def test_compact_matches_the_oracle(codec, n_slots):
    rng = np.random.default_rng(n_slots)
    B = 6
    lens = rng.integers(0, min(n_slots // 2, 300) * 16 // B + 1, B).tolist()
    other = W.FP8_E4M3 if codec != W.FP8_E4M3 else W.FP16
    s = table_case(B, 16, 64, lens, {codec: n_slots, other: 400}, n_slots + codec)
    check_compact(s, s["pools"][0])


def test_compact_full_empty_and_outside_holders():
    s = table_case(2, 16, 64, [512, 512], {W.FP16: 64}, 1, shared=0)
    assert check_compact(s, s["pools"][0]) == []                     # every slot is live
    s = table_case(2, 16, 64, [0, 0], {W.FP16: 64}, 1)
    assert check_compact(s, s["pools"][0]) == []                     # none is
    s["refs"][W.FP16][[3, 40, 63]] = [1, 2, -4]                      # held outside the table; a negative count is none
    assert check_compact(s, s["pools"][0]) == [(3, 0), (40, 1)]
    s["table"][0, :3], s["lens"][0] = [40, -1, 64], 40               # entries that name no slot stay and are counted
    check_compact(s, s["pools"][0])


def test_both_on_another_stream_and_from_a_graph():
    s = table_case(12, 16, 16, [100, 31, 7, 200, 0, 64, 65, 90, 16, 1, 222, 40], {W.BF16: 300, W.INT8: 300}, 9)
    parents, n_new = [3, 1, -1, 3, 0, 5, 6, 6, 8, 9, 10, 2], [1, 5, 3, 17, 2, 16, 0, 1, 1, 1, 9, 30]
    ref = run_fork(s, parents, n_new, W.BF16)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = run_fork(s, parents, n_new, W.BF16, stream=st)
    for x, y in zip(ref[:3], got[:3]):
        assert np.array_equal(x, y)
    t = torch.empty((12, 16), dtype=torch.int32, device=DEV)
    c = torch.empty((12, 16), dtype=torch.uint8, device=DEV)
    n = torch.empty(12, dtype=torch.int32, device=DEV)
    rin = [dev(s["refs"][p.codec]) for p in s["pools"]]
    rout = [torch.empty_like(r) for r in rin]
    rend, tend = torch.empty_like(rin[0]), torch.empty_like(t)
    live = torch.zeros(1, dtype=torch.int32, device=DEV)
    ins = [dev(np.array(x, np.int32)) for x in (parents, n_new)] + [dev(s["codec"]), dev(s["table"]), dev(s["lens"])]
    ws = torch.empty(argus.fork_workspace_bytes(12, s["pools"]), dtype=torch.uint8, device=DEV)
    ws2 = torch.empty(argus.compact_workspace_bytes(s["pools"][0]), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        argus.fork_pages(s["g"], ins[0], ins[1], W.BF16, s["pools"], rin, rout, ins[2], ins[3], ins[4], c, t, n, 16, ws)
        argus.compact_pages(s["g"], s["pools"][0], rout[0], rend, c, t, n, tend, 16, live, ws2)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(t.cpu().numpy(), ref[0]) and np.array_equal(rout[0].cpu().numpy(), ref[3][W.BF16])
        ot, orf, _, ol, _ = oracle.compact_pages(W.BF16, ref[3][W.BF16], ref[1], ref[0], ref[2], 16)
        assert np.array_equal(tend.cpu().numpy(), ot) and np.array_equal(rend.cpu().numpy(), orf) and int(live) == ol


def test_offsets_beyond_four_gigabytes():
    """A pool of 5 GB: a page forked and one compacted at its far end."""
    Hkv, P, D = 8, 16, 128
    page = 2 * Hkv * P * D * 2
    n = (5 << 30) // page + 3
    g = argus.geom(Hkv, Hkv, D, P)
    pool = argus.Pool(W.FP16, torch.empty((n, 2, Hkv, P, D), dtype=torch.float16, device=DEV), None, n)
    pool.codes[n - 2] = W.normal((2, Hkv, P, D), W.FP16, 1).to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    ref = torch.ones(n, dtype=torch.int32, device=DEV)
    ref[n - 1] = 0
    t, c, l = torch.empty((2, 1), dtype=torch.int32, device=DEV), torch.empty((2, 1), dtype=torch.uint8, device=DEV), i32([0, 0])
    r = torch.empty_like(ref)
    ws = torch.empty(argus.fork_workspace_bytes(2, [pool]), dtype=torch.uint8, device=DEV)
    argus.fork_pages(g, i32([0, 0]), i32([1, 1]), W.FP16, [pool], [ref], [r], torch.zeros((2, 1), dtype=torch.uint8, device=DEV),
                     i32([[n - 2], [-1]]), i32([5, 0]), c, t, l, 1, ws)
    assert t.tolist() == [[n - 2], [n - 1]] and torch.equal(pool.codes[n - 1], pool.codes[n - 2])
    assert r[n - 2:].tolist() == [1, 1]
    r.zero_()
    r[n - 1] = 2
    out, t2, live = torch.empty_like(r), torch.empty_like(t), torch.empty(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(argus.compact_workspace_bytes(pool), dtype=torch.uint8, device=DEV)
    argus.compact_pages(g, pool, r, out, c, t, l, t2, 1, live, ws)
    assert int(live) == 1 and out[0] == 2 and t2[1, 0] == 0 and torch.equal(pool.codes[0], pool.codes[n - 1])
