"""argus_attn_weights on the GPU against the double-precision oracle.

Bound per position: each weight 2^(s - L) is off by ln 2 times what its score is off by (D products summed in fp32, at
most D roundings of 2^-23 of the sum of their magnitudes; its scaling and the difference with L, 2^-22 of
|s| + |L|), and 2^x by 2^-21; the sum over n rows and the old weight adds at most (n + 2) 2^-24 of
the whole.
"""

import numpy as np
import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus
from mixed_precision_paged_argus_gb300 import workloads as W
import oracle
from test_gpu_extend import DEV, F8, I8, make, spoil_tails

pytestmark = pytest.mark.gpu
GROUPS = [W.INT4_G32, W.INT2_G32, W.INT1_G32]


def log_sums(c, causal):
    """Every row's log-sum by the oracle, as the attention would have left it."""
    q64 = c.to64(W.to_bits(c.q))
    return oracle.paged_extend(q64, c.q_start, c.Hkv, c.P, c.opools, c.page_codec, c.table, c.lens, c.scale, causal)[1].astype(np.float32)


def args_of(c, lse, causal=True, q=None, status=None):
    return argus.extend_args(c.g, c.q if q is None else q, torch.from_numpy(c.q_start).to(DEV), c.pools, c.d_codec, c.d_table, c.d_lens,
                             c.max_pages, c.scale, None, causal=causal, lse2_out=lse, status=status)


def check(c, causal=True, decay=0.5, row_extra=0, expect_bad=0, status=None, q=None):
    lse = log_sums(c, causal)
    old = np.random.default_rng(1).random((len(c.lens), c.Hkv, c.max_pages * c.P + row_extra)).astype(np.float32)
    got = torch.from_numpy(old).to(DEV)
    if decay == 0:
        got.fill_(float("nan"))                          # not read
    argus.attn_weights(args_of(c, torch.from_numpy(lse).to(DEV), causal, q, status), got, decay)
    torch.cuda.synchronize()
    ref, bad, err = oracle.attn_weights(c.to64(W.to_bits(c.q)), c.q_start, lse, c.Hkv, c.P, c.opools, c.page_codec, c.table, c.lens,
                                        c.scale, old.astype(np.float64), float(np.float32(decay)), causal)
    assert bad == expect_bad
    got = got.cpu().numpy().astype(np.float64)
    rows = np.diff(c.q_start).max() * (c.Hq // c.Hkv)
    for b, n in enumerate(c.lens):
        n = min(int(n), c.max_pages * c.P)
        bound = 2 * err[b, :, :n] + (rows + 2) * 2.0 ** -24 * np.abs(ref[b, :, :n])
        over = np.abs(got[b, :, :n] - ref[b, :, :n]) - bound
        assert not np.isnan(got[b, :, :n]).any() and (n == 0 or over.max() <= 0), over.max()
        if decay:
            assert np.array_equal(got[b, :, n:], old[b, :, n:].astype(np.float64))
        else:
            assert np.isnan(got[b, :, n:]).all()
    return got


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,codecs", [
    (W.FP16, [W.FP16]), (W.BF16, [W.BF16]), (W.FP16, [F8]), (W.BF16, [F8]), (W.FP16, [I8]), (W.BF16, [I8]), (W.FP16, GROUPS[:1]),
    (W.BF16, GROUPS[1:]), (W.FP16, [W.FP16, F8, I8] + GROUPS), (W.BF16, [W.BF16, F8, I8] + GROUPS)])
def test_tiers_types_and_masks(dtype, codecs, D, causal):
    c = make(8, 2, D, 16, [300, 17, 128, 129, 1], [5, 17, 1, 33, 1], codecs, dtype, seed=11 + D)
    if not set(codecs) & set(GROUPS):
        spoil_tails(c)
    check(c, causal, decay=0.5 if causal else 0.0, row_extra=5)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (9, 3), (8, 2), (10, 2), (12, 2), (14, 2), (16, 2)])
@pytest.mark.parametrize("n_q", [1, 2, 7, 40])
def test_head_groupings_and_row_counts(Hq, Hkv, n_q):
    c = make(Hq, Hkv, 64, 48, [200, 95, 500], [n_q, 3, max(1, n_q - 1)], [W.FP16, F8], W.FP16, seed=40 + Hq)
    spoil_tails(c)
    check(c, decay=1.0)


@pytest.mark.parametrize("n_q", [1, 16, 17, 33, 70, 150])
@pytest.mark.parametrize("dtype,codecs", [(W.BF16, [F8]), (W.BF16, [W.BF16, I8]), (W.FP16, [W.FP16])])
def test_many_rows(n_q, dtype, codecs):
    c = make(4, 1, 128, 32, [257, 700], [n_q, max(1, n_q - 1)], codecs, dtype, seed=70 + n_q)
    spoil_tails(c)
    check(c, decay=0.9)


@pytest.mark.parametrize("new", [[1, 1, 1], [3, 2, 0], [6, 5, 4], [21, 1, 1], [9, 1, 0], [1, 30, 2]])
@pytest.mark.parametrize("dtype,codecs", [(W.FP16, [W.FP16, W.INT4_G32, F8]), (W.BF16, [W.BF16, W.INT2_G32, I8])])
def test_uneven_rows_over_group_codes(new, dtype, codecs):
    """Odd and even numbers of tiles of eight rows, a sequence without rows beside one of many."""
    c = make(8, 2, 128, 32, [257, 700, 40], new, codecs, dtype, seed=75)
    check(c, decay=0.9)


@pytest.mark.parametrize("length", [1, 15, 16, 17, 127, 128, 129, 511, 512, 513, 1025])
def test_lengths_around_the_chunks(length):
    for new in (1, min(70, length)):
        c = make(4, 2, 64, 16, [length, 3], [new, 1], [I8], W.FP16, seed=100 + length)
        spoil_tails(c)
        check(c)


def test_sequences_that_see_nothing_or_ask_nothing():
    c = make(4, 2, 128, 16, [0, 40, 3, 0, 50], [2, 0, 7, 0, 20], [F8], W.BF16, seed=130)
    got = check(c, decay=0.25)
    assert got[1, :, :40].max() <= 0.25
    check(c, decay=0.0)
    c = make(4, 2, 64, 16, [5, 40], [0, 0], [F8], W.FP16, seed=131)
    check(c, decay=0.5)


def test_the_weights_of_a_row_sum_to_one():
    """With the attention's own log-sums."""
    from test_gpu_extend import run
    c = make(16, 2, 128, 64, [4000, 777], [3, 64], [W.BF16, F8, I8], W.BF16, seed=140)
    _, lse = run(c, True)
    w = torch.zeros((2, 2, c.max_pages * 64), device=DEV)
    argus.attn_weights(args_of(c, lse), w)
    assert torch.allclose(w.double().sum(-1), torch.tensor([[24.0] * 2, [512.0] * 2], dtype=torch.float64, device=DEV), rtol=1e-5)


def test_after_decode():
    from paged_cases import run_decode
    c = make(32, 4, 128, 64, [1000, 64, 777], [1, 1, 1], [W.BF16, F8, I8, W.INT4_G32], W.BF16, seed=150)
    lse = run_decode(c, out_dtype=torch.bfloat16)[2]
    w = torch.zeros((3, 4, c.max_pages * 64), device=DEV)
    argus.attn_weights(args_of(c, lse), w, 0.0)
    for b, n in enumerate((1000, 64, 777)):
        assert torch.allclose(w[b, :, :n].double().sum(-1), torch.full((4,), 8.0, dtype=torch.float64, device=DEV), rtol=1e-4)
        assert torch.all(w[b, :, n:] == 0)


def test_bad_slots_and_missing_pools_add_nothing():
    c = make(4, 2, 64, 16, [400, 130], [30, 2], [F8, I8], W.FP16, seed=170)
    c.table[0, 3], c.table[0, 9], c.table[1, 8] = -1, 10000, -5
    c.page_codec[0, 5], c.page_codec[1, 2], c.page_codec[1, 3] = W.INT4_G32, W.FP16, 200
    c.d_table, c.d_codec = torch.from_numpy(c.table).to(DEV), torch.from_numpy(c.page_codec).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    check(c, expect_bad=6, status=status)
    assert int(status) == 6


def test_large_scores_and_scales():
    c = make(8, 2, 128, 16, [600], [6], [F8, I8], W.BF16, seed=151)
    rng = np.random.default_rng(5)
    for pool in c.pools:
        _, meta = c.opools[pool.codec]
        meta[:, 0] *= 2.0 ** rng.integers(0, 7, size=meta[:, 0].shape)
        meta[1::4, 0] = 0
        pool.meta.copy_(torch.from_numpy(meta))
    check(c)


@pytest.mark.parametrize("n_q", [2, 40])
def test_nan_queries_stay_in_their_sequence_and_head(n_q):
    c = make(8, 2, 64, 16, [300, 90], [n_q, 5], [F8], W.FP16, seed=175)
    lse = torch.from_numpy(log_sums(c, True)).to(DEV)
    clean, got = (torch.zeros((2, 2, c.max_pages * 16), device=DEV) for _ in range(2))
    argus.attn_weights(args_of(c, lse), clean)
    c.q[1, 6, 7] = float("nan")
    argus.attn_weights(args_of(c, lse), got)
    assert torch.isnan(got[0, 1, :300 - n_q + 2]).all() and torch.equal(got[0, 0], clean[0, 0]) and torch.equal(got[1], clean[1])


def test_strided_queries_other_rows_and_repeats():
    c = make(8, 2, 128, 16, [100, 300], [3, 9], [F8], W.BF16, seed=180)
    lse = torch.from_numpy(log_sums(c, True)).to(DEV)
    wide = torch.full((14, 12, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:12, 1:9] = c.q
    outs = []
    for q, L in ((c.q, lse), (wide[:, 1:9], torch.cat([lse, lse[:2] * float("nan")])), (c.q, lse)):
        w = torch.zeros((2, 2, c.max_pages * 16), device=DEV)
        argus.attn_weights(args_of(c, L.contiguous(), q=q), w)
        outs.append(w)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_many_sequences():
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 200, 700).tolist()
    new = [int(rng.integers(0, min(n, 4) + 1)) for n in lens]
    check(make(4, 2, 64, 16, lens, new, [W.FP16, I8], W.FP16, seed=190))


def test_replayed_from_a_graph_with_other_lengths():
    c = make(8, 2, 128, 16, [2000, 333, 64], [4, 20, 64], [W.BF16, F8], W.BF16, seed=220)
    lse = torch.from_numpy(log_sums(c, True)).to(DEV)
    w = torch.zeros((3, 2, c.max_pages * 16), device=DEV)
    args = args_of(c, lse)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        argus.attn_weights(args, w, 0.5)
    for lens in ([2000, 333, 64], [1999, 200, 64]):
        c.lens = np.array(lens)
        c.d_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        new_lse = log_sums(c, True)
        lse.copy_(torch.from_numpy(new_lse))
        w.fill_(0.125)
        graph.replay()
        torch.cuda.synchronize()
        ref, _, err = oracle.attn_weights(c.to64(W.to_bits(c.q)), c.q_start, new_lse, c.Hkv, c.P, c.opools, c.page_codec, c.table, c.lens, c.scale,
                                          np.full(tuple(w.shape), 0.125), 0.5)
        assert np.all(np.abs(w.cpu().numpy() - ref) <= 2 * err + 258 * 2.0 ** -24 * np.abs(ref))


@pytest.mark.parametrize("n_q", [1, 40])
def test_offsets_beyond_four_gigabytes(n_q):
    small = make(16, 8, 128, 16, [77, 160], [n_q, 2], [F8], W.BF16, seed=520)
    lse = torch.from_numpy(log_sums(small, True)).to(DEV)
    ref, got = (torch.zeros((2, 8, small.max_pages * 16), device=DEV) for _ in range(2))
    argus.attn_weights(args_of(small, lse), ref)
    n = (5 << 30) // (2 * 8 * 16 * 128)
    codes, meta = torch.empty((n, 2, 8, 16, 128), dtype=torch.uint8, device=DEV), torch.empty((n, 2, 8), device=DEV)
    pool = small.pools[0]
    codes[-pool.n_slots:], meta[-pool.n_slots:] = pool.codes, pool.meta
    small.pools = [argus.Pool(F8, codes, meta, n)]
    small.d_table = small.d_table + (n - pool.n_slots)
    argus.attn_weights(args_of(small, lse), got)
    assert torch.equal(ref, got)


@pytest.mark.parametrize("seed", range(10))
def test_random_batches(seed):
    rng = np.random.default_rng(3000 + seed)
    B, Hkv, G = int(rng.integers(1, 9)), int(rng.integers(1, 4)), int(rng.integers(1, 9))
    D, P, dtype = int(rng.choice([64, 128])), int(rng.choice([16, 32, 48, 80])), int(rng.choice([W.FP16, W.BF16]))
    lens = [int(x) for x in rng.integers(0, 700, B)]
    new = [int(rng.integers(0, min(90, n + 3) + 1)) for n in lens]
    c = make(G * Hkv, Hkv, D, P, lens, new, [c for c in (dtype, F8, I8, *GROUPS) if rng.random() < 0.5] or [F8], dtype, seed=300 + seed)
    if int(c.q_start[-1]) == 0:
        return
    check(c, bool(rng.integers(0, 2)), float(rng.choice([0.0, 0.7, 1.0])))


def test_one_sequence_asks_for_all():
    """No more tokens than sequences, all of one: its many rows go through the kernel of decode steps."""
    for n_q in (5, 30):
        c = make(8, 2, 128, 16, [200] + [40, 0, 17] * 10, [n_q] + [0] * 30, [F8, W.BF16], W.BF16, seed=192)
        spoil_tails(c)
        check(c, decay=0.5)


@pytest.mark.parametrize("L,n_q,codec", [(300000, 1, F8), (100000, 32, F8), (70000, 40, W.BF16), (300000, 1, W.BF16)])
def test_long_sequences(L, n_q, codec):
    """More chunks and blocks per warp and CTA than are looked up at once; against a dense computation in 64 bits."""
    Hq, Hkv, D, P = 16, 8, 128, 64
    pages = -(-L // P)
    gen = torch.Generator(device=DEV).manual_seed(L + n_q)
    rand = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    if codec == F8:
        codes = (rand(pages, 2, Hkv, P, D) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        meta = 0.008 + 0.004 * torch.rand((pages, 2, Hkv), generator=gen, device=DEV)
    else:
        codes, meta = rand(pages, 2, Hkv, P, D).bfloat16(), None
    pool = argus.Pool(codec, codes, meta, pages)
    q = rand(n_q, Hq, D).bfloat16()
    table = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)[None].contiguous()
    args_of_ = lambda lse: argus.extend_args(  # noqa: E731
        argus.geom(Hq, Hkv, D, P), q, torch.tensor([0, n_q], dtype=torch.int32, device=DEV), [pool],
        torch.full((1, pages), codec, dtype=torch.uint8, device=DEV), table, torch.tensor([L], dtype=torch.int32, device=DEV), pages, D ** -0.5, None,
        lse2_out=lse)
    ref, bound = torch.empty((Hkv, L), dtype=torch.float64, device=DEV), torch.empty((Hkv, L), dtype=torch.float64, device=DEV)
    lse = torch.empty((n_q, Hq), device=DEV)
    see = torch.arange(L, device=DEV)[None] <= L - n_q + torch.arange(n_q, device=DEV)[:, None]
    for h in range(Hkv):
        k = codes[table[0].long(), 0, h]
        k = (k.view(torch.float8_e4m3fn).double() * meta[table[0].long(), 0, h].double()[:, None, None] if codec == F8 else k.double()).reshape(-1, D)[:L]
        x = torch.einsum("ngd,kd->gnk", q[:, 2 * h:2 * h + 2].double(), k) * (D ** -0.5 * 1.4426950408889634)
        mag = torch.einsum("ngd,kd->gnk", q[:, 2 * h:2 * h + 2].double().abs(), k.abs()) * (D ** -0.5 * 1.4426950408889634)
        x = x.masked_fill(~see, -float("inf"))
        L2 = torch.logsumexp(x * 0.6931471805599453, -1) * 1.4426950408889634
        lse[:, 2 * h:2 * h + 2] = L2.t().float()
        p = torch.exp2(x - lse[:, 2 * h:2 * h + 2].t().double()[..., None])
        ref[h] = p.sum((0, 1))
        e = 0.6931471805599453 * (D * 2.0 ** -23 * mag + 2.0 ** -22 * (x.abs().nan_to_num(posinf=0.0) + L2.abs()[..., None])) + 2.0 ** -21
        bound[h] = (2 * p * e).sum((0, 1))
    w = torch.full((1, Hkv, pages * P), 0.25, device=DEV)
    argus.attn_weights(args_of_(lse), w, 0.5)
    got = w[0, :, :L].double() - 0.125
    assert torch.all((got - ref).abs() <= bound + (2 * n_q + 2) * 2.0 ** -24 * (ref + 0.125))
    assert torch.all(w[0, :, L:] == 0.25)
