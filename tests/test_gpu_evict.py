"""argus_evict_tokens on the GPU against the oracle: what is kept, its weights, and the new pages' codes and scales,
all bit for bit."""

import numpy as np
import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus
from mixed_precision_paged_argus_gb300 import workloads as W
import oracle
from oracle import codecs as C
from test_gpu_extend import DEV, F8, I8, make, spoil_tails

pytestmark = pytest.mark.gpu
GROUPS = [W.INT4_G32, W.INT2_G32, W.INT1_G32]


def weights(c, seed, extra=0, ties=True):
    rng = np.random.default_rng(seed)
    w = np.exp(2 * rng.standard_normal((len(c.lens), c.Hkv, c.max_pages * c.P + extra))).astype(np.float32)
    if ties:
        w = np.round(w * 4) / 4                          # many share a value, many are 0
    return w.astype(np.float32)


class Evicted:
    pass


def call(c, w, budget, sinks, recent, codec, dst_pages=None, extra_out=3, status=None, dst=None, stream=None):
    e = Evicted()
    B = len(c.lens)
    e.pages = max(1, -(-budget // c.P)) if dst_pages is None else dst_pages
    e.n_slots = B * e.pages + 3
    e.table = np.random.default_rng(9).permutation(e.n_slots)[:B * e.pages].reshape(B, e.pages).astype(np.int32)
    e.dst = argus.Pool.empty(codec, e.n_slots, c.Hkv, c.P, c.D, device=DEV) if dst is None else dst
    e.dst.codes.view(torch.uint8).fill_(0x3C)
    if e.dst.meta is not None:
        e.dst.meta.fill_(7.0)
    e.lens = torch.full((B,), -5, dtype=torch.int32, device=DEV)
    e.kept = torch.full((B, c.Hkv, budget), -5, dtype=torch.int32, device=DEV)
    e.w = torch.full((B, c.Hkv, budget + extra_out), float("nan"), device=DEV)
    argus.evict_tokens(c.g, c.pools, c.d_codec, c.d_table, c.d_lens, c.max_pages, torch.from_numpy(w).to(DEV), budget, sinks, recent, e.dst,
                       torch.from_numpy(e.table).to(DEV), e.pages, e.lens, e.kept, e.w, status=status, stream=stream)
    torch.cuda.synchronize()
    return e


def check(c, w, budget, sinks, recent, codec, **kw):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    e = call(c, w, budget, sinks, recent, codec, status=status, **kw)
    codes, meta = C.alloc_pool(codec, e.n_slots, c.Hkv, c.P, c.D)
    codes.view(np.uint8)[...] = 0x3C
    if meta is not None:
        meta[...] = 7.0
    lens, kept, w_out, bad = oracle.evict_tokens(c.Hkv, c.P, c.D, c.opools, c.page_codec, c.table, c.lens, w, budget, sinks, recent, codec, codes, meta,
                                                 e.table, e.w.shape[2])
    assert np.array_equal(e.lens.cpu().numpy(), lens)
    assert np.array_equal(e.kept.cpu().numpy(), kept)
    assert np.array_equal(e.w.cpu().numpy().view(np.int32), w_out.view(np.int32))
    got = e.dst.codes.cpu().view(torch.int16 if codec <= W.BF16 else torch.uint8).numpy().astype(np.int64)
    want = (codes.view(np.int16) if codec <= W.BF16 else codes.view(np.uint8)).astype(np.int64)
    # -0 (an e4m3 code, which the oracle's table of values gives as 0) and 0 are the same value
    minus = {F8: 0x80, I8: None}.get(codec, -0x8000)
    got, want = np.where(got == minus, 0, got) if minus is not None else got, np.where(want == minus, 0, want) if minus is not None else want
    assert np.array_equal(got, want)
    if meta is not None:
        assert np.array_equal(e.dst.meta.cpu().numpy(), meta)
    assert int(status) == bad
    return e, bad


@pytest.mark.parametrize("D,P", [(64, 16), (128, 16), (128, 64), (64, 48), (64, 160)])
@pytest.mark.parametrize("dtype,codecs,to", [
    (W.FP16, [W.FP16], W.FP16), (W.BF16, [W.BF16], W.BF16), (W.FP16, [F8], F8), (W.BF16, [I8], I8), (W.BF16, [W.BF16, F8, I8], W.BF16),
    (W.FP16, [W.FP16, F8, I8], F8), (W.FP16, [W.FP16, F8] + GROUPS, W.FP16), (W.BF16, [I8] + GROUPS, I8), (W.FP16, GROUPS, F8), (W.FP16, GROUPS, W.BF16)])
def test_tiers_and_new_pages(dtype, codecs, to, D, P):
    c = make(6, 3, D, P, [500, 90, 231, 17, 1, 0], [1] * 6, codecs, dtype, seed=D + P + to)
    check(c, weights(c, 1, extra=2), 100, 4, 30, to)


@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (16, 4, 12), (17, 0, 0), (64, 64, 0), (64, 0, 64), (299, 1, 1), (300, 4, 4),
                                                 (400, 0, 0), (33, 3, 5)])
def test_budgets(budget, sinks, recent):
    c = make(4, 2, 64, 16, [300, 301, 64, 33, 0], [1] * 5, [W.FP16], W.FP16, seed=budget)
    e, _ = check(c, weights(c, budget), budget, sinks, recent, W.FP16)
    assert torch.all(e.lens <= budget)


def test_a_budget_of_nothing():
    c = make(4, 2, 64, 16, [300, 0], [1, 1], [W.FP16], W.FP16, seed=3)
    e = call(c, weights(c, 2), 0, 0, 0, W.FP16)
    assert torch.all(e.lens == 0) and torch.all(e.w == 0)
    assert torch.all(e.dst.codes.view(torch.uint8) == 0x3C)


@pytest.mark.parametrize("kind", ["equal", "zero", "signs", "nan", "inf", "subnormal", "last_bit"])
def test_orders_of_weights(kind):
    """Ties go to the lower position; NaN counts below all else, -0 as 0."""
    c = make(2, 2, 64, 16, [700, 64], [1, 1], [W.FP16], W.FP16, seed=5)
    rng = np.random.default_rng(6)
    w = np.full((2, 2, c.max_pages * 16), 0.25, np.float32)
    if kind == "zero":
        w = np.where(rng.random(w.shape) < 0.5, 0.0, -0.0)
    elif kind == "signs":
        w = rng.integers(-3, 4, w.shape) * 0.5
    elif kind == "nan":
        w = np.where(rng.random(w.shape) < 0.95, np.nan, rng.integers(-1, 2, w.shape))
    elif kind == "inf":
        w = rng.choice([np.inf, -np.inf, 1.0, np.nan, 3e38], w.shape)
    elif kind == "subnormal":
        w = rng.integers(-2, 3, w.shape) * 1e-45
    elif kind == "last_bit":
        w = (np.float32(1.0).view(np.int32) + rng.integers(0, 2, w.shape)).astype(np.int32).view(np.float32)
    w = np.ascontiguousarray(w.astype(np.float32))
    for budget in (40, 333):
        e = call(c, w, budget, 4, 10, W.FP16)
        for b, L in enumerate((700, 64)):
            for h in range(2):
                ks = oracle.evict_keep(w[b, h], L, budget, 4, 10)
                assert e.kept[b, h, :len(ks)].tolist() == ks


@pytest.mark.parametrize("L", [1000, 1024, 1025, 32767, 32768, 32769, 70000, 262144, 262145, 400000])
def test_long_rows(L):
    """One block, clusters of 2 to 8, and rows that are read again in every round."""
    P, D, Hkv = 1024, 64, 2
    pages = -(-L // P)
    pool = argus.Pool.empty(F8, 1, Hkv, P, D, device=DEV, zero=True)
    g = argus.geom(4, Hkv, D, P)
    w = torch.rand((2, Hkv, pages * P), device=DEV)
    w = torch.where(w < 0.3, 0.25, w)
    lens = torch.tensor([L, max(1, L // 3)], dtype=torch.int32, device=DEV)
    budget, sinks, recent = 700, 5, 100
    kept, lens_out = torch.empty((2, Hkv, budget), dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)
    w_out = torch.empty((2, Hkv, budget), device=DEV)
    dst = argus.Pool.empty(F8, 2, Hkv, P, D, device=DEV)
    for _ in range(2):
        argus.evict_tokens(g, [pool], torch.full((2, pages), F8, dtype=torch.uint8, device=DEV), torch.zeros((2, pages), dtype=torch.int32, device=DEV),
                           lens, pages, w, budget, sinks, recent, dst, torch.arange(2, dtype=torch.int32, device=DEV)[:, None].contiguous(), 1,
                           lens_out, kept, w_out)
        for b, n in enumerate(lens.tolist()):
            m = min(n, budget)
            assert int(lens_out[b]) == m
            for h in range(Hkv):
                x = w[b, h, :n].double().cpu()
                if n > budget:
                    x[:sinks], x[n - recent:] = 9.0, 9.0
                    order = torch.sort(x, descending=True, stable=True).indices[:budget].sort().values
                else:
                    order = torch.arange(n)
                assert torch.equal(kept[b, h, :m].cpu().long(), order)
                assert torch.equal(w_out[b, h, :m].cpu(), w[b, h].cpu()[order])
        w = -torch.log(w + 1e-3)                         # the range wanders, negative values among them


@pytest.mark.parametrize("bits", [6, 10, 14])
def test_many_weights_that_differ_in_their_last_bits(bits):
    """More keys share their first bits than the late rounds' list holds."""
    rng = np.random.default_rng(40 + bits)
    c = make(2, 1, 64, 64, [20000, 5000], [1, 1], [W.FP16], W.FP16, seed=40)
    w = (np.float32(1.0).view(np.int32) + rng.integers(0, 1 << bits, (2, 1, c.max_pages * c.P), dtype=np.int32)).view(np.float32)
    w[0, 0, 5000:5030] = -w[0, 0, 5000:5030]
    for budget in (1, 333, 4999):
        check(c, w, budget, 1 if budget > 1 else 0, 0, W.FP16)


@pytest.mark.parametrize("extra", [0, 1, 2, 130, 5003])
def test_weights_behind_the_kept_ones_are_cleared(extra):
    c = make(4, 2, 64, 16, [700, 0, 33, 50], [1, 1, 1, 1], [W.FP16], W.FP16, seed=44)
    for budget in (0, 1, 50, 64):
        w = weights(c, 45)
        if budget:
            check(c, w, budget, 0, 0, W.FP16, extra_out=extra)
        elif extra:
            assert not call(c, w, 0, 0, 0, W.FP16, extra_out=extra).w.any()


def test_pages_without_a_place():
    c = make(4, 2, 64, 16, [400, 130], [1, 1], [F8, I8], W.FP16, seed=170)
    c.table[0, 3], c.table[0, 0], c.table[1, 8] = -1, 10000, -5
    c.page_codec[0, 5], c.page_codec[1, 2], c.page_codec[1, 3] = W.INT4_G32, W.FP16, 200
    c.d_table, c.d_codec = torch.from_numpy(c.table).to(DEV), torch.from_numpy(c.page_codec).to(DEV)
    _, bad = check(c, weights(c, 4), 120, 8, 40, F8)
    assert bad > 0
    _, bad = check(c, weights(c, 4), 120, 8, 40, W.FP16)
    assert bad > 0


@pytest.mark.parametrize("to", [W.FP16, F8])
def test_new_pages_that_are_not_there(to):
    c = make(4, 2, 64, 32, [400, 130, 20], [1, 1, 1], [F8], W.FP16, seed=171)
    w = weights(c, 5)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    e = call(c, w, 100, 4, 10, to)
    table = torch.from_numpy(e.table).to(DEV)
    table[0, 1], table[1, 3], table[2, 1] = -1, e.n_slots, -1      # the last one is not used
    whole = e.dst.codes.clone()
    e.dst.codes.view(torch.uint8).fill_(0x11)
    argus.evict_tokens(c.g, c.pools, c.d_codec, c.d_table, c.d_lens, c.max_pages, torch.from_numpy(w).to(DEV), 100, 4, 10, e.dst, table, e.pages, e.lens,
                       e.kept, e.w, status=status)
    assert int(status) == 2
    lost = {int(e.table[0, 1]), int(e.table[1, 3])}
    used = [int(e.table[b, j]) for b, n in ((0, 4), (1, 4), (2, 1)) for j in range(n)]
    for s in range(e.n_slots):
        if s in used and s not in lost:
            assert torch.equal(e.dst.codes[s], whole[s])
        else:
            assert torch.all(e.dst.codes[s].view(torch.uint8) == 0x11)


def test_into_the_same_pool():
    """The new pages may lie in the pool that the old ones are read from."""
    c = make(8, 2, 128, 16, [600, 333], [1, 1], [F8], W.BF16, seed=172, extra_slots=30)
    w = weights(c, 6)
    ref, _ = check(c, w, 200, 4, 50, F8)
    pool = c.pools[0]
    free = torch.tensor(sorted(set(range(pool.n_slots)) - set(c.table[0, :38].tolist()) - set(c.table[1, :21].tolist()))[:26], dtype=torch.int32)
    table = free.view(2, 13).to(DEV)
    lens, kept, w_out = torch.empty_like(ref.lens), torch.empty_like(ref.kept), torch.empty_like(ref.w)
    old = pool.codes.clone()
    argus.evict_tokens(c.g, c.pools, c.d_codec, c.d_table, c.d_lens, c.max_pages, torch.from_numpy(w).to(DEV), 200, 4, 50, pool, table, 13, lens, kept, w_out)
    assert torch.equal(kept, ref.kept)
    for b in range(2):
        for j in range(13):
            assert torch.equal(pool.codes[int(table[b, j])], ref.dst.codes[int(ref.table[b, j])])
            assert torch.equal(pool.meta[int(table[b, j])], ref.dst.meta[int(ref.table[b, j])])
    rest = torch.ones(pool.n_slots, dtype=torch.bool, device=DEV)
    rest[table.flatten().long()] = False
    assert torch.equal(pool.codes[rest], old[rest])


def test_magnitudes_and_zero_pages():
    c = make(4, 2, 64, 16, [300], [1], [F8, I8], W.FP16, seed=173)
    rng = np.random.default_rng(7)
    for pool in c.pools:
        _, meta = c.opools[pool.codec]
        meta *= 2.0 ** rng.integers(-60, 60, size=meta.shape)
        meta[::3] = 0
        pool.meta.copy_(torch.from_numpy(meta))
    for to in (F8, I8):
        check(c, weights(c, 7), 120, 0, 40, to)


def test_a_graph_on_another_stream():
    c = make(8, 2, 128, 16, [2000, 333, 64], [1, 1, 1], [W.BF16, F8], W.BF16, seed=220)
    w = weights(c, 8)
    ref = call(c, w, 500, 4, 100, F8)
    out = [torch.zeros_like(x) for x in (ref.lens, ref.kept, ref.w)]
    dst = argus.Pool.empty(F8, ref.n_slots, c.Hkv, c.P, c.D, device=DEV)
    t, wd = torch.from_numpy(ref.table).to(DEV), torch.from_numpy(w).to(DEV)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        argus.evict_tokens(c.g, c.pools, c.d_codec, c.d_table, c.d_lens, c.max_pages, wd, 500, 4, 100, dst, t, ref.pages, out[0], out[1], out[2])
    for _ in range(2):
        dst.codes.view(torch.uint8).fill_(0x3C)
        dst.meta.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], ref.lens) and torch.equal(out[1], ref.kept) and torch.equal(out[2], ref.w)
        assert torch.equal(dst.codes, ref.dst.codes) and torch.equal(dst.meta, ref.dst.meta)
    c.d_lens.copy_(torch.tensor([499, 0, 64], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert out[0].tolist() == [499, 0, 64] and out[1][0, 0, :499].tolist() == list(range(499))


def test_offsets_beyond_four_gigabytes():
    c = make(16, 8, 128, 16, [300, 160], [1, 1], [F8], W.BF16, seed=520)
    w = weights(c, 9)
    ref = call(c, w, 100, 4, 20, W.BF16)
    n = (5 << 30) // (2 * 8 * 16 * 128)
    codes, meta = torch.empty((n, 2, 8, 16, 128), dtype=torch.uint8, device=DEV), torch.empty((n, 2, 8), device=DEV)
    pool = c.pools[0]
    codes[-pool.n_slots:], meta[-pool.n_slots:] = pool.codes, pool.meta
    c.pools = [argus.Pool(F8, codes, meta, n)]
    c.d_table = c.d_table + (n - pool.n_slots)
    dst = torch.empty((n // 2,) + tuple(ref.dst.codes.shape[1:]), dtype=torch.bfloat16, device=DEV)
    t = torch.from_numpy(ref.table).to(DEV) + (n // 2 - ref.n_slots)
    out = [torch.zeros_like(x) for x in (ref.lens, ref.kept, ref.w)]
    argus.evict_tokens(c.g, c.pools, c.d_codec, c.d_table, c.d_lens, c.max_pages, torch.from_numpy(w).to(DEV), 100, 4, 20, argus.Pool(W.BF16, dst, None, n // 2),
                       t, ref.pages, out[0], out[1], out[2])
    torch.cuda.synchronize()
    assert torch.equal(out[1], ref.kept)
    used = torch.from_numpy(ref.table).long().flatten().to(DEV)
    assert torch.equal(dst[used + (n // 2 - ref.n_slots)], ref.dst.codes[used])


@pytest.mark.parametrize("seed", range(8))
def test_random_batches(seed):
    rng = np.random.default_rng(4000 + seed)
    B, Hkv = int(rng.integers(1, 7)), int(rng.integers(1, 4))
    D, P, dtype = int(rng.choice([64, 128])), int(rng.choice([16, 32, 80, 256])), int(rng.choice([W.FP16, W.BF16]))
    lens = [int(x) for x in rng.integers(0, 600, B)]
    c = make(Hkv, Hkv, D, P, lens, [1] * B, [c for c in (dtype, F8, I8, *GROUPS) if rng.random() < 0.5] or [F8], dtype, seed=300 + seed)
    spoil = {p.codec for p in c.pools} <= {dtype, F8, I8}
    if spoil:
        spoil_tails(c)
    budget = int(rng.integers(1, 500))
    sinks = int(rng.integers(0, min(budget, 20) + 1))
    check(c, weights(c, seed, ties=seed % 2 == 0), budget, sinks, int(rng.integers(0, budget - sinks + 1)), int(rng.choice([dtype, F8, I8])))
