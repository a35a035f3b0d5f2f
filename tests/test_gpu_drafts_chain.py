"""The operators of drafted trees and short caches as a server uses them: a prompt appended with normed heads, drafted
trees attended, their accepted paths moved, weights of what the queries looked at summed, sequences evicted to a budget,
decoded and extended from there -- every attention against a dense computation in 64 bits that keeps each KV head's rows
by itself and knows nothing of pages."""

import math

import numpy as np
import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus
from mixed_precision_paged_argus_gb300 import workloads as W
import oracle
from oracle import codecs as C

pytestmark = pytest.mark.gpu
DEV = "cuda"
Hq, Hkv, D, P, MAXP, ROWS = 8, 2, 64, 16, 20, 3
G, HALF, EPS = Hq // Hkv, 16, 1e-5


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def to64(x):
    return C.bf16_bits_to_f64(W.to_bits(x.contiguous()))


class Server:
    def __init__(self):
        self.g = argus.geom(Hq, Hkv, D, P)
        n = ROWS * MAXP
        self.pool, self.pool8 = (argus.Pool.empty(c, n, Hkv, P, D, device=DEV, zero=True) for c in (W.BF16, W.FP8_E4M3))
        perm = np.random.default_rng(0).permutation(n).reshape(ROWS, MAXP).astype(np.int32)
        self.table, self.codec = torch.from_numpy(perm).to(DEV), torch.full((ROWS, MAXP), W.BF16, dtype=torch.uint8, device=DEV)
        self.lens = i32([0] * ROWS)
        self.inv = torch.tensor([100.0 ** (-i / HALF) for i in range(HALF)], dtype=torch.float64, device=DEV)
        rng = np.random.default_rng(1)
        self.wq, self.wk = ((1 + 0.2 * rng.standard_normal(D)).astype(np.float32) for _ in range(2))
        self.weights = torch.zeros((ROWS, Hkv, MAXP * P), device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        # per row and KV head: keys and values in float64, as stored, and the weight that each position has
        self.k = [[[] for _ in range(Hkv)] for _ in range(ROWS)]
        self.v = [[[] for _ in range(Hkv)] for _ in range(ROWS)]
        self.w = [[[] for _ in range(Hkv)] for _ in range(ROWS)]

    def append(self, new, seed, depth=None):
        """New tokens for every row; depth: each token's position behind the row's end (a tree's), else in order."""
        self.new = new
        self.lens = self.lens + i32(new)
        self.q_start = i32([0] + np.cumsum(new).tolist())
        total = sum(new)
        qkv = W.normal((total, Hq + 2 * Hkv, D), W.BF16, seed).to(DEV)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        lens = self.lens.tolist()
        pos = np.concatenate([lens[b] - n + np.array(depth[b] if depth else np.arange(n)) for b, n in enumerate(new)]).astype(np.int32)[None]
        self.q = torch.empty((total, Hq, D), dtype=torch.bfloat16, device=DEV)
        argus.norm_rope_append(self.g, q, k, v, self.q, self.q_start, self.lens, torch.from_numpy(pos).to(DEV), self.inv, self.pool, self.codec,
                               self.table, MAXP, torch.from_numpy(self.wq).to(DEV), torch.from_numpy(self.wk).to(DEV), EPS, status=self.status)
        assert int(self.status) == 0
        ref_k = oracle.rotate(oracle.head_norm(to64(k), self.wk, EPS), pos, self.inv.cpu().numpy(), None, False)
        ref_q = oracle.rotate(oracle.head_norm(to64(q), self.wq, EPS), pos, self.inv.cpu().numpy(), None, False)
        # half a step, doubled for the oracle's and the kernel's value on two sides of a rounding border
        assert np.abs(to64(self.q) - ref_q).max() <= 2 * 2.0 ** -8 * np.abs(ref_q).max()
        table, t = self.table.cpu().numpy(), 0
        for b, n in enumerate(new):
            for i in range(n):
                at = lens[b] - n + i
                row = to64(self.pool.codes[int(table[b, at // P]), :, :, at % P])
                assert np.abs(row[0] - ref_k[t]).max() <= 2 * 2.0 ** -8 * np.abs(ref_k[t]).max()
                for h in range(Hkv):
                    self.k[b][h].append(row[0, h])
                    self.v[b][h].append(row[1, h])
                    self.w[b][h].append(0.0)
                t += 1

    def attend(self, call, sees):
        """call(args, ws); sees(b, i, n, L, pos).  Checked against the dense computation."""
        out, self.lse = torch.empty_like(self.q), torch.empty((self.q.shape[0], Hq), device=DEV)
        self.args = argus.extend_args(self.g, self.q, self.q_start, [self.pool, self.pool8], self.codec, self.table, self.lens, MAXP,
                                      1.0 / math.sqrt(D), out, lse2_out=self.lse, status=self.status)
        call(self.args, torch.empty(argus.extend_workspace_bytes(self.args), dtype=torch.uint8, device=DEV))
        torch.cuda.synchronize()
        assert int(self.status) == 0
        q64, got, t = to64(self.q), out.float().cpu().numpy(), 0
        for b, n in enumerate(self.new):
            for i in range(n):
                for h in range(Hq):
                    k, v = np.array(self.k[b][h // G]), np.array(self.v[b][h // G])
                    keep = sees(b, i, n, len(k), np.arange(len(k)))
                    s = k[keep] @ q64[t, h] / math.sqrt(D)
                    w = np.exp(s - s.max())
                    lse = (s.max() + math.log(w.sum())) / math.log(2)
                    w /= w.sum()
                    ref, av = w @ v[keep], w @ np.abs(v[keep])
                    # p and the result rounded to bf16 once each; scores of a few units in fp32
                    assert np.all(np.abs(got[t, h] - ref) <= 2.0 ** -8 * (av + np.abs(ref)) + 1e-4 * av + 1e-30)
                    assert abs(float(self.lse[t, h]) - lse) <= 1e-4
                t += 1

    def weigh(self, decay):
        """What causal attention of the newest queries looked at."""
        argus.attn_weights(self.args, self.weights, decay)
        q64, got, t = to64(self.q), self.weights.cpu().numpy(), 0
        for b, n in enumerate(self.new):
            for h in range(Hkv):
                self.w[b][h] = [decay * x for x in self.w[b][h]]
            for i in range(n):
                L = len(self.k[b][0])
                see = L - n + i + 1
                for h in range(Hq):
                    s = np.array(self.k[b][h // G])[:see] @ q64[t, h] / math.sqrt(D) / math.log(2)
                    for j, x in enumerate(2.0 ** (s - float(self.lse[t, h]))):
                        self.w[b][h // G][j] += x
                t += 1
            for h in range(Hkv):
                ref = np.array(self.w[b][h])
                # every weight to 1e-5 of itself: scores of a few units, some of their 24 bits lost
                assert np.all(np.abs(got[b, h, :len(ref)] - ref) <= 1e-5 * ref + 1e-9)
                self.w[b][h] = got[b, h, :len(ref)].astype(np.float64).tolist()

    def accept(self, paths):
        width = max(1, max(len(p) for p in paths))
        path = np.full((ROWS, width), -1, np.int32)
        for b, p in enumerate(paths):
            path[b, :len(p)] = p
        lens = torch.empty_like(self.lens)
        argus.accept_tokens(self.g, self.pool, self.codec, self.table, MAXP, self.q_start, self.lens, torch.from_numpy(path).to(DEV),
                            i32([len(p) for p in paths]), lens, status=self.status)
        for b, n in enumerate(self.new):
            base = len(self.k[b][0]) - n
            for h in range(Hkv):
                for x in (self.k, self.v, self.w):
                    x[b][h] = x[b][h][:base] + [x[b][h][base + i] for i in paths[b]]
        self.lens = lens
        assert int(self.status) == 0 and lens.tolist() == [len(k[0]) for k in self.k]

    def evict(self, budget, sinks, recent, codec):
        dst = {W.BF16: self.pool, W.FP8_E4M3: self.pool8}[codec]
        pages = -(-budget // P)
        used = set(self.table.flatten().tolist())
        if codec == W.BF16:
            # the pools have a page for every entry: new ones go where no row's length reaches
            reach = [-(-int(n) // P) for n in self.lens]
            used = {int(self.table[b, j]) for b in range(ROWS) for j in range(reach[b])}
        free = [s for s in range(dst.n_slots) if s not in used] if codec == W.BF16 else list(range(dst.n_slots))
        to = np.array(free[:ROWS * pages], np.int32).reshape(ROWS, pages)
        lens, kept, w = torch.empty_like(self.lens), torch.empty((ROWS, Hkv, budget), dtype=torch.int32, device=DEV), torch.empty_like(self.weights)
        argus.evict_tokens(self.g, [self.pool, self.pool8], self.codec, self.table, self.lens, MAXP, self.weights, budget, sinks, recent, dst,
                           torch.from_numpy(to).to(DEV), pages, lens, kept, w, status=self.status)
        torch.cuda.synchronize()
        assert int(self.status) == 0
        kept = kept.cpu().numpy()
        rest = [s for s in range(ROWS * MAXP) if codec == W.FP8_E4M3 or s not in set(to.flatten().tolist())]
        for b in range(ROWS):
            L = len(self.k[b][0])
            for h in range(Hkv):
                ks = oracle.evict_keep(np.array(self.w[b][h], np.float32), L, budget, sinks, recent)
                assert kept[b, h, :len(ks)].tolist() == ks
                for x in (self.k, self.v, self.w):
                    x[b][h] = [x[b][h][j] for j in ks]
        self.lens, self.weights = lens, w
        assert lens.tolist() == [len(k[0]) for k in self.k]
        # the new table: the new pages, then 16-bit ones that nobody uses for what is appended
        table, codecs = np.full((ROWS, MAXP), -1, np.int32), np.full((ROWS, MAXP), W.BF16, np.uint8)
        table[:, :pages], codecs[:, :pages] = to, codec
        spare = iter(rest)
        for b in range(ROWS):
            m = -(-int(lens[b]) // P)
            for j in range(m, MAXP):
                table[b, j], codecs[b, j] = next(spare, -1), W.BF16
        self.table, self.codec = torch.from_numpy(table).to(DEV), torch.from_numpy(codecs).to(DEV)
        for b in range(ROWS):
            for j in range(len(self.k[b][0])):
                slot = int(table[b, j // P])
                if codec == W.BF16:
                    x, small = to64(self.pool.codes[slot, :, :, j % P]), 0.0
                else:
                    meta = self.pool8.meta[slot].cpu().double().numpy()
                    x = self.pool8.codes[slot, :, :, j % P].cpu().view(torch.float8_e4m3fn).double().numpy() * meta[..., None]
                    small = 2.0 ** -10 * meta.max()      # half of e4m3's smallest step
                for h in range(Hkv):
                    # half a step of the new type (and the scale's fp32 rounding); exact where the old page was of it
                    half = (2.0 ** -8 if codec == W.BF16 else 2.0 ** -4) * 1.001
                    for i, mine in enumerate((self.k, self.v)):
                        assert np.all(np.abs(x[i, h] - mine[b][h][j]) <= half * np.abs(mine[b][h][j]) + small)
                        mine[b][h][j] = x[i, h]


def tree_of(n, seed):
    rng = np.random.default_rng(seed)
    par = [-1] + [int(rng.integers(-1, i)) for i in range(1, n)]
    masks, depth = [], []
    for i, a in enumerate(par):
        masks.append(1 << i | (masks[a] if a >= 0 else 0))
        depth.append(0 if a < 0 else depth[a] + 1)
    return masks, depth


def path_of(masks, leaf):
    return [i for i in range(len(masks)) if masks[leaf] >> i & 1]


def test_a_servers_steps():
    s = Server()
    causal = lambda b, i, n, L, pos: pos <= L - n + i  # noqa: E731
    s.append([120, 37, 200], 1)
    s.attend(argus.paged_extend_attn, causal)
    s.weigh(0.0)
    for step in range(2):
        # drafted trees, attended, and the path of one leaf accepted
        trees = [tree_of(n, 10 * step + n) for n in (12, 33, 1)]
        s.append([12, 33, 1], 2 + step, depth=[d for _, d in trees])
        masks = torch.from_numpy(np.array([[m & 0xFFFFFFFF, m >> 32] for t, _ in trees for m in t], np.uint32).view(np.int32)).to(DEV)
        s.attend(lambda args, ws: argus.paged_tree_attn(args, ws, masks), oracle.tree_sees([t for t, _ in trees]))
        s.accept([path_of(t, len(t) - 1) for t, _ in trees])
    # one token each under a window, then causally, and its weights
    s.append([1, 1, 1], 5)
    s.attend(lambda args, ws: argus.paged_window_extend_attn(args, ws, 50, 4), oracle.window_sees(50, 4))
    s.attend(argus.paged_extend_attn, causal)
    s.weigh(0.5)
    s.evict(32, 4, 10, W.FP8_E4M3)                       # full pages: new tokens go to 16-bit ones
    s.append([20, 3, 1], 6)
    s.attend(argus.paged_extend_attn, causal)
    s.weigh(1.0)
    s.evict(34, 2, 10, W.BF16)                           # ends within a page, or keeps a shorter row whole
    s.append([1, 5, 9], 7)
    s.attend(lambda args, ws: argus.paged_window_extend_attn(args, ws, 30, 1), oracle.window_sees(30, 1))


def test_calls_on_two_streams_at_once():
    """Every operator on two streams together, with outputs (and workspaces) of their own: the bits of calls one by one."""
    from test_gpu_evict import call as evict, weights as some_weights
    from test_gpu_extend import make
    from test_gpu_masks import args_of, tree, words_of

    def steps(seed):
        c = make(8, 2, 128, 16, [900, 40, 333], [9, 40, 33], [W.BF16, W.FP8_E4M3], W.BF16, seed=seed)
        mask = words_of([tree(n, n) for n in c.new], 2)
        results = []

        def run(stream):
            args, ws, out, lse = args_of(c)
            args2, ws2, out2, lse2 = args_of(c)
            w = torch.zeros((3, 2, c.max_pages * 16), device=DEV)
            torch.cuda.synchronize()
            for _ in range(3):
                argus.paged_window_extend_attn(args, ws, 100, 4, stream=stream)
                argus.paged_tree_attn(args2, ws2, mask, stream=stream)
                argus.attn_weights(args, w, 0.0, stream=stream)
            return out, lse, out2, lse2, w
        return c, run, results

    cases = [steps(900), steps(901)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    alone = []
    for c, run, _ in cases:
        got = run(torch.cuda.current_stream())
        torch.cuda.synchronize()
        alone.append([x.clone() for x in got])
    together = [run(s) for (_, run, _), s in zip(cases, streams)]
    torch.cuda.synchronize()
    for a, t in zip(alone, together):
        for x, y in zip(a, t):
            assert torch.equal(x, y)
    refs = [evict(c, some_weights(c, 3), 200, 4, 50, W.FP8_E4M3) for c, _, _ in cases]
    for s, (c, _, _), r in zip(streams, cases, refs):
        e = evict(c, some_weights(c, 3), 200, 4, 50, W.FP8_E4M3, stream=s)
        assert torch.equal(e.kept, r.kept) and torch.equal(e.w, r.w) and torch.equal(e.dst.meta, r.dst.meta) and torch.equal(e.dst.codes, r.dst.codes)
