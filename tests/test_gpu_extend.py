"""argus_paged_extend_attn on the GPU against the double-precision oracle.

Bound per output element, from the arithmetic (u = eps / 2 of the 16-bit type, a
rounding to nearest): every p_j is rounded once to that type for P.V, the
result once for the output; a score sums D exact products in fp32 (at most D
roundings of 2^-23 of the sum of their magnitudes, truncating adds included), and 2^x
is off by 2^-21 plus the fp32 rounding of x, in the numerator and in the sum:
  |o - ref| <= u sum p|v| + u |ref| + 2 e sum p|v|,  e = ln 2 (D 2^-23 qk + 2^-22 smax) + 2^-21
(plus the output type's smallest step).  Where P is fp16 (an fp16 query, or 8-bit pages
alone) it is stored relative to a reference that its largest p_j s_j (s_j: the page's V
scale) does not lie below, times 2^7: so the largest stored P is at least 2^7, and a P in fp16's
subnormal range (step 2^-24) is off by at most 2^-25 = 2^-32 of the largest:
  + 2^-32 max_j (p_j s_j) sum_j |code_j| / sum p.
"""

import math

import numpy as np
import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus
from mixed_precision_paged_argus_gb300 import workloads as W
import oracle
from oracle import codecs as C
from paged_cases import DEV, build_case

pytestmark = pytest.mark.gpu
F8, I8 = W.FP8_E4M3, W.INT8


def make(Hq, Hkv, D, P, lens, new, codecs, dtype, seed, extra_slots=2):
    """A paged case with new[b] query tokens for sequence b; codecs: the choices of
    each page's tier."""
    rng = np.random.default_rng(seed)
    max_pages = max(1, max((n + P - 1) // P for n in lens))
    pc = rng.choice(codecs, size=(len(lens), max_pages))
    c = build_case(Hq, Hkv, D, P, lens, pc, dtype, seed=seed, extra_slots=extra_slots)
    c.new = list(new)
    c.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    total = int(c.q_start[-1])
    c.q = W.normal((total, Hq, D), dtype, seed + 50).to(DEV)
    c.dtype = dtype
    c.to64 = C.f16_bits_to_f64 if dtype == W.FP16 else C.bf16_bits_to_f64
    return c


def spoil_tails(c):
    """Rows of each last page behind the sequence's end: NaN (0x7F bytes) in the GPU's pools."""
    by = {p.codec: p for p in c.pools}
    for b, n in enumerate(c.lens):
        page = int(n) // c.P
        for p in range(page, c.max_pages):
            pool = by[int(c.page_codec[b, p])]
            pool.codes.view(torch.uint8)[int(c.table[b, p]), :, :, (int(n) - p * c.P if p == page else 0):] = 0x7F


def run(c, causal, q=None, status=None, stream=None, ws=None, max_pages=None):
    q = c.q if q is None else q
    out = torch.full((q.shape[0], c.Hq, c.D), float("nan"), dtype=q.dtype, device=DEV)
    lse = torch.full((q.shape[0], c.Hq), float("nan"), dtype=torch.float32, device=DEV)
    args = argus.extend_args(c.g, q, torch.from_numpy(c.q_start).to(DEV), c.pools, c.d_codec, c.d_table, c.d_lens,
                             c.max_pages, c.scale, out, causal=causal, lse2_out=lse, status=status)
    if ws is None:
        ws = torch.full((argus.extend_workspace_bytes(args),), 0xFF, dtype=torch.uint8, device=DEV)
    argus.paged_extend_attn(args, ws, stream=stream)
    torch.cuda.synchronize()
    return out, lse


def check(c, out, lse, causal, expect_bad=0, rows=None):
    q64 = c.to64(W.to_bits(c.q))
    ref, ref_lse, bad, av, pc, qk, smax = oracle.paged_extend(q64, c.q_start, c.Hkv, c.P, c.opools, c.page_codec, c.table,
                                                          c.lens, c.scale, causal)
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
    # lse2 in bits: the score's error, the sum's and log2's (2^-21 relative each), and its own fp32 rounding
    lb = c.D * 2.0 ** -23 * qk + 2.0 ** -22 * smax + 2.0 ** -19 + 2.0 ** -22 * np.abs(np.where(fin, ref_lse, 0))
    assert np.all(np.abs(gl[fin] - ref_lse[fin]) <= lb[fin])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,codecs", [
    (W.FP16, [W.FP16]), (W.BF16, [W.BF16]), (W.FP16, [F8]), (W.BF16, [F8]), (W.FP16, [I8]), (W.BF16, [I8]),
    (W.FP16, [W.FP16, F8, I8]), (W.BF16, [W.BF16, F8, I8])])
def test_tiers_types_and_masks(dtype, codecs, D, causal):
    c = make(8, 2, D, 16, [300, 17, 128, 129, 1], [5, 17, 1, 33, 1], codecs, dtype, seed=11 + D)
    spoil_tails(c)
    out, lse = run(c, causal)
    check(c, out, lse, causal)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (9, 3), (8, 2), (10, 2), (12, 2), (14, 2), (16, 2)])
def test_head_groupings(Hq, Hkv):
    c = make(Hq, Hkv, 64, 48, [200, 95, 500], [40, 3, 70], [W.FP16, F8], W.FP16, seed=40 + Hq)
    spoil_tails(c)
    out, lse = run(c, True)
    check(c, out, lse, True)


@pytest.mark.parametrize("n_q", [1, 2, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 130])
def test_row_counts_around_the_tiles(n_q):
    """n_q * G rows: 4 to 520, around the 32, 64 and 128 rows where the layout changes."""
    c = make(4, 1, 128, 32, [257, 700], [n_q, max(1, n_q - 1)], [W.BF16, F8], W.BF16, seed=70 + n_q)
    out, lse = run(c, True)
    check(c, out, lse, True)


@pytest.mark.parametrize("length", [1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1025])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths_around_the_blocks(length, causal):
    c = make(4, 2, 64, 16, [length], [min(3, length)], [I8], W.FP16, seed=100 + length)
    spoil_tails(c)
    out, lse = run(c, causal)
    check(c, out, lse, causal)


def test_rows_that_see_nothing():
    """An empty cache, a sequence without queries, and a causal batch with more queries than positions."""
    c = make(4, 2, 128, 16, [0, 40, 3, 0], [2, 0, 7, 0], [F8], W.BF16, seed=130)
    for causal in (True, False):
        out, lse = run(c, causal)
        check(c, out, lse, causal)
        assert torch.all(out[:2] == 0) and torch.all(torch.isinf(lse[:2]))
    out, lse = run(c, True)
    assert torch.all(out[2:6] == 0) and torch.all(torch.isinf(lse[2:6])) and torch.all(torch.isfinite(lse[6:]))


def test_rows_of_no_sequence_are_left():
    c = make(4, 2, 64, 16, [40, 90], [3, 5], [W.FP16], W.FP16, seed=140)
    total = 8
    c.q = torch.cat([c.q, torch.full((4, 4, 64), float("nan"), dtype=torch.float16, device=DEV)])
    out, lse = run(c, True)
    assert torch.isnan(out[total:]).all() and torch.isnan(lse[total:]).all()
    c.q, out, lse = c.q[:total], out[:total], lse[:total]
    check(c, out, lse, True)


def test_large_scores_and_scale_ranges():
    """Scores of hundreds (the running maximum moves far), pages whose V scales differ by 2^40 or are 0."""
    c = make(8, 2, 128, 16, [600], [6], [F8, I8], W.BF16, seed=150)
    rng = np.random.default_rng(5)
    for pool in c.pools:
        codes, meta = c.opools[pool.codec]
        meta[:, 1] *= 2.0 ** rng.integers(-20, 21, size=meta[:, 1].shape)
        meta[::3, 1] = 0
        meta[:, 0] *= 2.0 ** rng.integers(0, 7, size=meta[:, 0].shape)
        meta[1::4, 0] = 0
        pool.meta.copy_(torch.from_numpy(meta))
    out, lse = run(c, True)
    check(c, out, lse, True)


def test_a_softmax_scale_of_zero_averages():
    c = make(4, 1, 64, 16, [77], [4], [W.FP16], W.FP16, seed=160)
    c.scale = 0.0
    out, lse = run(c, True)
    check(c, out, lse, True)
    assert torch.allclose(lse[3], torch.tensor(math.log2(77.0), device=DEV), atol=1e-5)


def test_bad_slots_and_missing_pools_are_left_out_and_counted():
    c = make(4, 2, 64, 16, [400, 130], [70, 2], [F8, I8], W.FP16, seed=170)
    c.table[0, 3], c.table[0, 9], c.table[1, 8] = -1, 10000, -5       # the last one is the partial last page
    c.page_codec[0, 5] = W.INT4_G32
    c.page_codec[1, 2] = W.BF16                                       # no such pool in the call
    c.page_codec[1, 3] = 200
    c.d_table, c.d_codec = torch.from_numpy(c.table).to(DEV), torch.from_numpy(c.page_codec).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = run(c, True, status=status)
    check(c, out, lse, True, expect_bad=6)
    assert int(status) == 6


@pytest.mark.parametrize("dtype,codec", [(W.FP16, W.FP16), (W.BF16, F8)])
def test_nan_queries_stay_in_their_rows(dtype, codec):
    """A query row that holds NaN gives NaN, also where its item is cut over many CTAs, and leaves the
    tile's other rows alone."""
    c = make(4, 1, 64, 16, [20000, 90, 0], [5, 40, 3], [codec], dtype, seed=175)
    clean, clean_lse = run(c, True)
    c.q[2, 1, 7] = c.q[20, 3, 63] = c.q[46, 0, 0] = float("nan")      # the last one's cache is empty
    out, lse = run(c, True)
    hit = torch.zeros(c.q.shape[:2], dtype=torch.bool, device=DEV)
    hit[2, 1] = hit[20, 3] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


@pytest.mark.parametrize("dtype,codecs", [(W.FP16, [F8]), (W.BF16, [F8]), (W.BF16, [W.BF16, F8])])
def test_nan_queries_do_not_reach_later_items(dtype, codecs):
    """Every CTA takes many items, long ones with NaN rows before short ones whose tiles hold fewer rows."""
    lens, new = [70, 40, 60, 33] * 200, [32, 3, 17, 1] * 200
    c = make(4, 1, 64, 16, lens, new, codecs, dtype, seed=176)
    clean, clean_lse = run(c, True)
    long = torch.from_numpy(np.repeat(np.array(new) > 16, new)).to(DEV)
    c.q[long] = float("nan")
    out, lse = run(c, True)
    assert torch.isnan(out[long]).all() and torch.isnan(lse[long]).all()
    assert torch.equal(out[~long], clean[~long]) and torch.equal(lse[~long], clean_lse[~long])


def test_strided_queries():
    c = make(8, 2, 128, 16, [100, 300], [3, 9], [F8], W.BF16, seed=180)
    wide = torch.full((12, 12, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 1:9] = c.q
    dense, dl = run(c, True)
    out, lse = run(c, True, q=wide[:, 1:9])
    assert torch.equal(out, dense) and torch.equal(lse, dl)


@pytest.mark.parametrize("batch", [40, 700])
def test_many_sequences(batch):
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 60, batch).tolist()
    new = [int(rng.integers(0, min(n, 4) + 1)) for n in lens]
    c = make(4, 2, 64, 16, lens, new, [W.FP16, I8], W.FP16, seed=190)
    out, lse = run(c, True)
    check(c, out, lse, True)


def test_one_token_equals_the_decode_call():
    from paged_cases import run_decode
    c = make(32, 4, 128, 64, [1000, 64, 777], [1, 1, 1], [W.BF16, F8, I8], W.BF16, seed=200)
    out, lse = run(c, True)
    check(c, out, lse, True)
    _, o32, dl, _ = run_decode(c, out_dtype=torch.bfloat16)
    # two roundings to bf16 apart (p and the output), each half a step of values up to sum p|v| <= max |v|
    assert (out.float() - o32).abs().max() <= 2 * 2.0 ** -8 * 6.0
    assert torch.allclose(lse, dl, atol=1e-4)


def test_a_long_chunk_at_sampled_rows():
    """600 new tokens over 9,000 cached ones, three tiers: rows checked at the ends and between."""
    c = make(16, 2, 128, 64, [9000], [600], [W.BF16, F8, I8], W.BF16, seed=210)
    out, lse = run(c, True)
    rows = [0, 1, 15, 16, 299, 583, 599]
    q64 = c.to64(W.to_bits(c.q))
    for t in rows:
        sub = np.array([0, 1])
        ref, rl, _, av, pc, qk, smax = oracle.paged_extend(q64[t:t + 1], sub, c.Hkv, c.P, c.opools, c.page_codec, c.table,
                                                       [9000 - 600 + t + 1], c.scale, True)
        e = (math.log(2) * (c.D * 2.0 ** -23 * qk + 2.0 ** -22 * smax) + 2.0 ** -21)[..., None]
        bound = 2.0 ** -8 * (av + np.abs(ref)) + 2 * e * av + 1e-38
        assert np.all(np.abs(out[t:t + 1].float().cpu().numpy() - ref) <= bound), t
        assert np.abs(lse[t:t + 1].cpu().numpy() - rl).max() <= 1e-3


def test_streams_graphs_and_repeats():
    """The same bits on another stream, from a captured graph with new inputs, and with a dirty workspace."""
    c = make(8, 2, 128, 16, [2000, 333, 64], [4, 20, 64], [W.BF16, F8], W.BF16, seed=220)
    ref, rl = run(c, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = run(c, True, stream=s)
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    args = argus.extend_args(c.g, c.q, torch.from_numpy(c.q_start).to(DEV), c.pools, c.d_codec, c.d_table, c.d_lens,
                             c.max_pages, c.scale, out, lse2_out=lse)
    ws = torch.empty(argus.extend_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    with torch.cuda.stream(s):
        argus.paged_extend_attn(args, ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        argus.paged_extend_attn(args, ws)
    for shift in (0, 1):
        if shift:      # other lengths in the same graph
            c.lens = np.array([1999, 200, 64])
            c.d_lens.copy_(torch.tensor([1999, 200, 64], dtype=torch.int32))
        out.fill_(float("nan"))
        lse.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        if not shift:
            assert torch.equal(out, ref) and torch.equal(lse, rl)
        check(c, out, lse, True)


@pytest.mark.parametrize("dtype,with16", [(W.FP16, False), (W.BF16, False), (W.BF16, True)])
@pytest.mark.parametrize("codec", [F8, I8])
@pytest.mark.parametrize("D", [64, 128])
def test_every_code_is_exact(D, codec, dtype, with16):
    """Sequences of one token: the output is that token's V, code times scale, rounded once.  Four sequences hold
    every code (without e4m3's NaN); with16: the call has a 16-bit page in the same block (bf16 operands)."""
    P, B = 16, 512 // D
    codes = np.arange(256, dtype=np.uint8)
    if codec == F8:
        codes[[0x7F, 0xFF]] = 0
    elif codec == I8:
        codes[0x80] = 0          # -128 is not a code
    pool = argus.Pool.empty(codec, B, 1, P, D, device=DEV, zero=True)
    pool.codes[:, 1, 0, 0] = torch.from_numpy(np.resize(codes, (B, D))).to(DEV)
    pool.meta.fill_(0.5)
    pools = [pool]
    table, pc = np.arange(B, dtype=np.int32)[:, None], np.full((B, 1), codec, np.uint8)
    if with16:                   # an empty 16-bit page in front: V = 0 and K = 0, so each of two keys weighs 1/2
        pools.append(argus.Pool.empty(dtype, 1, 1, P, D, device=DEV, zero=True))
        table, pc = np.concatenate([np.zeros_like(table), table], 1), np.concatenate([np.full_like(pc, dtype), pc], 1)
    lens = [P + 1 if with16 else 1] * B
    q = torch.ones((B, 1, D), dtype=torch.float16 if dtype == W.FP16 else torch.bfloat16, device=DEV)
    out = torch.empty_like(q)
    args = argus.extend_args(argus.geom(1, 1, D, P), q, torch.arange(B + 1, dtype=torch.int32, device=DEV), pools,
                             torch.from_numpy(pc).to(DEV), torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                             table.shape[1], 1.0, out)
    argus.paged_extend_attn(args, torch.empty(argus.extend_workspace_bytes(args), dtype=torch.uint8, device=DEV))
    v = torch.from_numpy(np.resize(codes, (B, D)))
    want = (v.view(torch.float8_e4m3fn).float() if codec == F8 else v.view(torch.int8).float()) * 0.5
    if with16:
        want = want / (P + 1)
    got = out[:, 0].float().cpu()
    # alone: exact but for the output's rounding; among P + 1 keys with p = 1: 1 / 17 in fp32 as well
    u = torch.finfo(out.dtype).eps / 2
    assert torch.all((got - want).abs() <= want.abs() * (u + 2.0 ** -21) + torch.finfo(out.dtype).smallest_normal * u)


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = np.random.default_rng(1000 + seed)
    B = int(rng.integers(1, 9))
    Hkv, G = int(rng.integers(1, 4)), int(rng.integers(1, 9))
    D, P = int(rng.choice([64, 128])), int(rng.choice([16, 32, 48, 80]))
    dtype = int(rng.choice([W.FP16, W.BF16]))
    lens = [int(x) for x in rng.integers(0, 700, B)]
    new = [int(rng.integers(0, min(90, n + 3) + 1)) for n in lens]
    codecs = [c for c in (dtype, F8, I8) if rng.random() < 0.6] or [F8]
    c = make(G * Hkv, Hkv, D, P, lens, new, codecs, dtype, seed=300 + seed)
    if int(c.q_start[-1]) == 0:
        return
    spoil_tails(c)
    for causal in (True, False):
        out, lse = run(c, causal)
        check(c, out, lse, causal)


def test_many_short_items_and_one_long():
    """The work list cuts long items and packs short ones: both in one call, causal and full."""
    c = make(8, 1, 64, 16, [6000] + [30] * 40, [40] + [30] * 40, [F8, W.FP16], W.FP16, seed=500)
    for causal in (True, False):
        out, lse = run(c, causal)
        check(c, out, lse, causal)


def test_two_streams_with_a_workspace_each():
    a = make(8, 2, 128, 16, [900, 40], [9, 40], [F8], W.BF16, seed=510)
    b = make(8, 2, 128, 16, [70, 1500], [1, 130], [I8, W.BF16], W.BF16, seed=511)
    refs = [run(c, True) for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls = []
    for c, s in zip((a, b), streams):
        out, lse = torch.full_like(c.q, float("nan")), torch.full(c.q.shape[:2], float("nan"), device=DEV)
        args = argus.extend_args(c.g, c.q, torch.from_numpy(c.q_start).to(DEV), c.pools, c.d_codec, c.d_table, c.d_lens,
                                 c.max_pages, c.scale, out, lse2_out=lse)
        calls.append((args, torch.empty(argus.extend_workspace_bytes(args), dtype=torch.uint8, device=DEV), s, out, lse))
    torch.cuda.synchronize()
    for _ in range(5):
        for args, ws, s, _, _ in calls:
            argus.paged_extend_attn(args, ws, stream=s)
    torch.cuda.synchronize()
    for (ref, rl), (_, _, _, out, lse) in zip(refs, calls):
        assert torch.equal(out, ref) and torch.equal(lse, rl)


def test_offsets_beyond_four_gigabytes():
    """Slots at the end of an FP8 pool of 5 GB, and query rows of a strided tensor."""
    Hkv, P, D = 8, 16, 128
    small = make(16, Hkv, D, P, [77, 160], [5, 2], [F8], W.BF16, seed=520)
    ref, rl = run(small, True)
    n_slots = (5 << 30) // (2 * Hkv * P * D)
    codes = torch.empty((n_slots, 2, Hkv, P, D), dtype=torch.uint8, device=DEV)
    meta = torch.empty((n_slots, 2, Hkv), dtype=torch.float32, device=DEV)
    pool = small.pools[0]
    codes[-pool.n_slots:], meta[-pool.n_slots:] = pool.codes, pool.meta
    small.pools = [argus.Pool(F8, codes, meta, n_slots)]
    small.d_table = small.d_table + (n_slots - pool.n_slots)
    out, lse = run(small, True)
    assert torch.equal(out, ref) and torch.equal(lse, rl)
