"""argus_paged_window_extend_attn and argus_paged_tree_attn on the GPU against the double-precision oracle.

The bounds are those of argus_paged_extend_attn (see test_gpu_extend.py): the kernels differ in what a
row sees alone.
"""

import math

import numpy as np
import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus
from mixed_precision_paged_argus_gb300 import workloads as W
import oracle
from test_gpu_extend import DEV, F8, I8, make, spoil_tails

pytestmark = pytest.mark.gpu


def tree(n, seed, words=None):
    """A random tree's masks: integers, and the rows of words."""
    rng = np.random.default_rng(seed)
    rows = []
    for i in range(n):
        a = int(rng.integers(-1, i)) if i else -1
        rows.append(1 << i | (rows[a] if a >= 0 else 0))
    return rows


def words_of(masks, words):
    rows = [[(x >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for m in masks for x in m]
    return torch.from_numpy(np.array(rows, np.uint32).reshape(-1, words).view(np.int32)).to(DEV)


def args_of(c, q=None, status=None):
    q = c.q if q is None else q
    out = torch.full((q.shape[0], c.Hq, c.D), float("nan"), dtype=q.dtype, device=DEV)
    lse = torch.full((q.shape[0], c.Hq), float("nan"), dtype=torch.float32, device=DEV)
    args = argus.extend_args(c.g, q, torch.from_numpy(c.q_start).to(DEV), c.pools, c.d_codec, c.d_table, c.d_lens, c.max_pages,
                             c.scale, out, lse2_out=lse, status=status)
    return args, torch.full((argus.extend_workspace_bytes(args),), 0xFF, dtype=torch.uint8, device=DEV), out, lse


def window(c, w, sinks, **kw):
    args, ws, out, lse = args_of(c, **kw)
    argus.paged_window_extend_attn(args, ws, w, sinks)
    torch.cuda.synchronize()
    return out, lse


def attend_tree(c, masks, words, **kw):
    args, ws, out, lse = args_of(c, **kw)
    argus.paged_tree_attn(args, ws, words_of(masks, words))
    torch.cuda.synchronize()
    return out, lse


def check(c, out, lse, sees, expect_bad=0):
    q64 = c.to64(W.to_bits(c.q))
    ref, ref_lse, bad, av, pc, qk, smax = oracle.paged_extend(q64, c.q_start, c.Hkv, c.P, c.opools, c.page_codec, c.table, c.lens,
                                                          c.scale, sees=sees)
    assert bad == expect_bad
    fi = torch.finfo(out.dtype)
    u = fi.eps / 2
    e = (math.log(2) * (c.D * 2.0 ** -23 * qk + 2.0 ** -22 * smax) + 2.0 ** -21)[..., None]
    got = out.float().cpu().numpy().astype(np.float64)
    bound = u * av + u * np.abs(ref) + 2 * e * av + fi.smallest_normal * fi.eps
    if c.dtype == W.FP16 or all(p.codec >= F8 for p in c.pools):
        bound = bound + 2.0 ** -32 * pc
    over = np.abs(got - ref) - bound
    assert not np.isnan(got).any() and over.max() <= 0, "worst %.3g over its bound" % over.max()
    gl = lse.cpu().numpy().astype(np.float64)
    fin = np.isfinite(ref_lse)
    assert np.array_equal(np.isfinite(gl), fin) and np.all(gl[~fin] == -np.inf)
    lb = c.D * 2.0 ** -23 * qk + 2.0 ** -22 * smax + 2.0 ** -19 + 2.0 ** -22 * np.abs(np.where(fin, ref_lse, 0))
    assert np.all(np.abs(gl[fin] - ref_lse[fin]) <= lb[fin])


@pytest.mark.parametrize("w,sinks", [(1, 0), (16, 4), (100, 0), (128, 128), (200, 130), (2 ** 31 - 1, 0), (5, 2 ** 31 - 1)])
@pytest.mark.parametrize("dtype,codecs,D", [(W.FP16, [W.FP16], 64), (W.BF16, [F8], 128), (W.BF16, [W.BF16, F8, I8], 128), (W.FP16, [I8], 64)])
def test_windows_types_and_tiers(dtype, codecs, D, w, sinks):
    c = make(8, 2, D, 16, [600, 17, 128, 400, 1], [5, 17, 1, 70, 1], codecs, dtype, seed=600 + D)
    spoil_tails(c)
    out, lse = window(c, w, sinks)
    check(c, out, lse, oracle.window_sees(w, sinks))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (9, 3), (10, 2), (14, 2), (16, 2)])
@pytest.mark.parametrize("w,sinks", [(130, 4), (256, 0)])
def test_windows_and_head_groupings(Hq, Hkv, w, sinks):
    """Many tiles per sequence: their blocks are counted in closed form."""
    c = make(Hq, Hkv, 64, 48, [900, 95, 1500], [140, 3, 210], [W.FP16, F8], W.FP16, seed=640 + Hq)
    spoil_tails(c)
    out, lse = window(c, w, sinks)
    check(c, out, lse, oracle.window_sees(w, sinks))


@pytest.mark.parametrize("Hq,Hkv", [(3, 1), (5, 1), (14, 2), (8, 1)])
@pytest.mark.parametrize("w,sinks", [(33, 36), (300, 516), (112, 16), (113, 113), (1, 129)])
def test_first_positions_that_end_inside_a_block(Hq, Hkv, w, sinks):
    """The window's chunks follow the first positions' in one block; tokens in front of the cache see nothing."""
    c = make(Hq, Hkv, 64, 16, [1900, 1153, 640, 90], [260, 33, 1, 200], [W.BF16, F8, I8], W.BF16, seed=645 + Hq)
    spoil_tails(c)
    out, lse = window(c, w, sinks)
    check(c, out, lse, oracle.window_sees(w, sinks))


def test_a_window_as_wide_as_the_cache_is_plain_attention():
    from test_gpu_extend import run
    c = make(8, 2, 128, 16, [700, 300], [40, 3], [W.BF16, F8], W.BF16, seed=650)
    plain = run(c, True)
    for w, sinks in ((700, 0), (1, 700), (2 ** 31 - 1, 2 ** 31 - 1)):
        got = window(c, w, sinks)
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])


def test_one_token_sees_what_decode_sees():
    from paged_cases import run_decode
    c = make(32, 4, 128, 64, [1000, 64, 777], [1, 1, 1], [W.BF16, F8, I8], W.BF16, seed=660)
    out, lse = window(c, 200, 4)
    _, o32, dl, _ = run_decode(c, out_dtype=torch.bfloat16, window=200, sinks=4)
    # two roundings to bf16 apart (p and the output), each half a step of values up to sum p|v| <= max |v|
    assert (out.float() - o32).abs().max() <= 2 * 2.0 ** -8 * 6.0
    assert torch.allclose(lse, dl, atol=1e-4)


def test_windows_where_the_cache_is_shorter_than_the_batch():
    c = make(4, 2, 128, 16, [0, 40, 3, 0], [2, 0, 7, 0], [F8], W.BF16, seed=670)
    out, lse = window(c, 2, 1)
    check(c, out, lse, oracle.window_sees(2, 1))
    assert torch.all(out[:6] == 0) and torch.all(torch.isinf(lse[:6])) and torch.all(torch.isfinite(lse[6:]))


def test_pages_out_of_sight_are_neither_read_nor_counted():
    c = make(4, 2, 64, 16, [800, 300], [3, 40], [F8, I8], W.FP16, seed=680)
    w, sinks = 100, 20
    sees = oracle.window_sees(w, sinks)
    for b, pages in ((0, [0, 1, 2, 30, 43, 44, 49]), (1, [5, 9, 18])):     # seen: 0, 1 (first tokens), 43 on; 10 on
        c.table[b, pages] = -1
    c.table[1, 12], c.page_codec[1, 13] = 10000, 200
    c.d_table, c.d_codec = torch.from_numpy(c.table).to(DEV), torch.from_numpy(c.page_codec).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = window(c, w, sinks, status=status)
    q64 = c.to64(W.to_bits(c.q))
    bad = oracle.paged_extend(q64, c.q_start, c.Hkv, c.P, c.opools, c.page_codec, c.table, c.lens, c.scale, sees=sees)[2]
    check(c, out, lse, sees, expect_bad=bad)
    assert int(status) == bad and bad >= 7


@pytest.mark.parametrize("P", [16, 48, 128, 1024])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_every_bad_page_in_sight_is_counted_once(P, G):
    """All pages bad, many tiles over them: each page that some token sees counts once."""
    n_new, L = 300, 2100
    c = make(G, 1, 64, P, [L, 50], [n_new, 50], [F8], W.FP16, seed=690)
    c.table[:] = -1
    c.d_table = torch.from_numpy(c.table).to(DEV)
    for w, sinks in ((1, 0), (40, 17), (333, 100), (5000, 0)):
        pos = np.arange(L)
        seen = (pos > L - n_new - w) | (pos < sinks)
        want = len(set(pos[seen] // P)) + len(set(np.arange(50) // P))
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out, lse = window(c, w, sinks, status=status)
        assert int(status) == want and torch.all(out == 0) and torch.all(lse == -math.inf)


@pytest.mark.parametrize("seed", range(10))
def test_random_windows(seed):
    rng = np.random.default_rng(2000 + seed)
    B, Hkv, G = int(rng.integers(1, 7)), int(rng.integers(1, 4)), int(rng.integers(1, 9))
    D, P, dtype = int(rng.choice([64, 128])), int(rng.choice([16, 32, 48, 80])), int(rng.choice([W.FP16, W.BF16]))
    lens = [int(x) for x in rng.integers(0, 900, B)]
    new = [int(rng.integers(0, min(90, n + 3) + 1)) for n in lens]
    c = make(G * Hkv, Hkv, D, P, lens, new, [c for c in (dtype, F8, I8) if rng.random() < 0.6] or [F8], dtype, seed=700 + seed)
    if int(c.q_start[-1]) == 0:
        return
    spoil_tails(c)
    w, sinks = int(rng.integers(1, 500)), int(rng.choice([0, 1, 64, 200]))
    out, lse = window(c, w, sinks)
    check(c, out, lse, oracle.window_sees(w, sinks))


@pytest.mark.parametrize("dtype,codecs,D", [(W.FP16, [W.FP16], 64), (W.BF16, [F8], 128), (W.BF16, [W.BF16, F8, I8], 128), (W.FP16, [I8], 64)])
@pytest.mark.parametrize("new", [[1, 5, 31], [32, 33, 64], [65, 130, 2]])
def test_trees_types_and_tiers(dtype, codecs, D, new):
    c = make(8, 2, D, 16, [300, 140, 70], new, codecs, dtype, seed=800 + D + new[0])
    spoil_tails(c)
    masks = [tree(n, 10 * n) for n in new]
    out, lse = attend_tree(c, masks, (max(new) + 31) // 32)
    check(c, out, lse, oracle.tree_sees(masks))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (9, 3), (10, 2), (14, 2)])
@pytest.mark.parametrize("base", [0, 1, 15, 16, 100, 127, 128, 129])
def test_trees_at_every_offset(Hq, Hkv, base):
    """The tree begins anywhere in a chunk or block of positions."""
    new = [40, 7]
    c = make(Hq, Hkv, 64, 32, [base + 40, base + 7], new, [W.FP16, F8], W.FP16, seed=820 + base)
    spoil_tails(c)
    masks = [tree(n, base + n) for n in new]
    out, lse = attend_tree(c, masks, 2)
    check(c, out, lse, oracle.tree_sees(masks))


def test_a_chain_is_causal_attention():
    from test_gpu_extend import run
    c = make(8, 2, 128, 16, [700, 300, 5], [40, 3, 5], [W.BF16, F8], W.BF16, seed=830)
    plain = run(c, True)
    masks = [[(1 << (i + 1)) - 1 for i in range(n)] for n in c.new]
    out, lse = attend_tree(c, masks, 2)
    check(c, out, lse, oracle.tree_sees(masks))
    check(c, *plain, oracle.tree_sees(masks))


def test_any_mask_is_taken():
    """Rows without a bit (the cache alone, or nothing where it is empty), bits of tokens that are not there, tokens
    without a word, more words than needed."""
    new = [40, 33, 3, 4]
    c = make(4, 2, 64, 16, [200, 33, 3, 2], new, [W.FP16, F8], W.FP16, seed=840)
    spoil_tails(c)
    rng = np.random.default_rng(1)
    masks = [[int(rng.integers(0, 2 ** 62)) for _ in range(n)] for n in new]
    masks[0][3] = masks[1][0] = masks[2][1] = 0
    for words in (1, 2, 5):
        seen = [[x & ((1 << 32 * words) - 1) for x in m] for m in masks]
        out, lse = attend_tree(c, seen, words)
        check(c, out, lse, oracle.tree_sees(seen))
        assert torch.all(out[40] == 0) and torch.all(lse[40] == -math.inf)


def test_bad_pages_under_a_tree_are_counted():
    c = make(4, 2, 64, 16, [400, 130], [70, 2], [F8, I8], W.FP16, seed=850)
    c.table[0, 3], c.table[0, 22], c.page_codec[1, 8] = -1, 10000, 200
    c.d_table, c.d_codec = torch.from_numpy(c.table).to(DEV), torch.from_numpy(c.page_codec).to(DEV)
    masks = [tree(n, n) for n in (70, 2)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = attend_tree(c, masks, 3, status=status)
    # the oracle counts the pages that are seen; those two and the last one are
    check(c, out, lse, oracle.tree_sees(masks), expect_bad=3)
    assert int(status) == 3


@pytest.mark.parametrize("kind", ["window", "tree"])
def test_rows_of_no_sequence_nan_queries_and_strides(kind):
    c = make(4, 2, 64, 16, [640, 90], [30, 5], [W.FP16, F8], W.FP16, seed=860)
    masks = [tree(n, n) for n in c.new]

    def call(q):
        extra = [[0] * (q.shape[0] - 35)] if q.shape[0] > 35 else []
        return window(c, 70, 3, q=q) if kind == "window" else attend_tree(c, masks + extra, 1, q=q)
    out, lse = call(c.q)
    wide = torch.full((35, 9, 64), float("nan"), dtype=torch.float16, device=DEV)
    wide[:, 3:7] = c.q
    got = call(wide[:, 3:7])
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    longer = torch.cat([c.q, c.q[:3]])
    longer[7, 2, 5] = float("nan")
    got = call(longer)
    assert torch.isnan(got[0][35:]).all() and torch.isnan(got[1][35:]).all()
    hit = torch.zeros((35, 4), dtype=torch.bool, device=DEV)
    hit[7, 2] = True
    assert torch.isnan(got[0][:35][hit]).all() and torch.equal(got[0][:35][~hit], out[~hit]) and torch.equal(got[1][:35][~hit], lse[~hit])


@pytest.mark.parametrize("kind", ["window", "tree"])
def test_replayed_from_a_graph_with_other_lengths(kind):
    c = make(8, 2, 128, 16, [2000, 333, 64], [4, 20, 64], [W.BF16, F8], W.BF16, seed=870)
    masks = [tree(n, n) for n in c.new]
    args, ws, out, lse = args_of(c)
    mask = words_of(masks, 2)
    sees = oracle.window_sees(90, 4) if kind == "window" else oracle.tree_sees(masks)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = (lambda **k: argus.paged_window_extend_attn(args, ws, 90, 4, **k)) if kind == "window" else (lambda **k: argus.paged_tree_attn(args, ws, mask, **k))
    call(stream=s)
    s.synchronize()
    check(c, out, lse, sees)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    for lens in ([2000, 333, 64], [1999, 200, 64]):
        c.lens = np.array(lens)
        c.d_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        lse.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(c, out, lse, sees)


def test_many_sequences_with_windows_and_trees():
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 300, 500).tolist()
    new = [int(rng.integers(0, min(n, 6) + 1)) for n in lens]
    c = make(4, 2, 64, 16, lens, new, [W.FP16, I8], W.FP16, seed=880)
    out, lse = window(c, 50, 4)
    check(c, out, lse, oracle.window_sees(50, 4))
    masks = [tree(n, 7 + n) for n in new]
    out, lse = attend_tree(c, masks, 1)
    check(c, out, lse, oracle.tree_sees(masks))


def test_a_long_chunk_under_a_window_at_sampled_rows():
    c = make(16, 2, 128, 64, [9000], [600], [W.BF16, F8, I8], W.BF16, seed=890)
    w, sinks = 1000, 70
    out, lse = window(c, w, sinks)
    q64 = c.to64(W.to_bits(c.q))
    for t in (0, 1, 15, 16, 299, 583, 599):
        L = 9000 - 600 + t + 1
        ref, rl, _, av, pc, qk, smax = oracle.paged_extend(q64[t:t + 1], np.array([0, 1]), c.Hkv, c.P, c.opools, c.page_codec, c.table, [L],
                                                       c.scale, sees=oracle.window_sees(w, sinks))
        e = (math.log(2) * (c.D * 2.0 ** -23 * qk + 2.0 ** -22 * smax) + 2.0 ** -21)[..., None]
        bound = 2.0 ** -8 * (av + np.abs(ref)) + 2 * e * av + 1e-38
        assert np.all(np.abs(out[t:t + 1].float().cpu().numpy() - ref) <= bound), t
        lb = c.D * 2.0 ** -23 * qk + 2.0 ** -22 * smax + 2.0 ** -19 + 2.0 ** -22 * np.abs(rl)
        assert np.all(np.abs(lse[t:t + 1].cpu().numpy() - rl) <= lb)
