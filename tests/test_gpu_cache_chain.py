"""The cache operators as a server uses them: prompts appended with their positions, attended, demoted, forked into
beams, extended by single tokens, compacted -- the attention of every step against a dense computation
in 64 bits that knows nothing of pages (the tokens' rotated keys and values as the library rounded them)."""

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
Hq, Hkv, D, P, MAXP = 8, 2, 64, 16, 12
HALF = 16


class Server:
    def __init__(self, rows, n_slots):
        self.g = argus.geom(Hq, Hkv, D, P)
        self.rows, self.n16, self.n8 = rows, n_slots, n_slots
        self.pool = argus.Pool.empty(W.BF16, n_slots, Hkv, P, D, device=DEV, zero=True)
        self.pool8 = argus.Pool.empty(W.FP8_E4M3, n_slots, Hkv, P, D, device=DEV, zero=True)
        self.table = torch.full((rows, MAXP), -1, dtype=torch.int32, device=DEV)
        self.codec = torch.zeros((rows, MAXP), dtype=torch.uint8, device=DEV)
        self.lens = torch.zeros(rows, dtype=torch.int32, device=DEV)
        self.ref = [torch.zeros(n_slots, dtype=torch.int32, device=DEV) for _ in range(2)]
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.inv = torch.tensor([100.0 ** (-i / HALF) for i in range(HALF)], dtype=torch.float64, device=DEV)
        self.axis = (torch.arange(HALF, device=DEV) % 3).to(torch.uint8)
        self.tokens = [([], []) for _ in range(rows)]      # per row: keys and values [Hkv][D] in float64, as stored

    def fork(self, parents, new):
        t, c, n = torch.empty_like(self.table), torch.empty_like(self.codec), torch.empty_like(self.lens)
        out = [torch.empty_like(r) for r in self.ref]
        pools = [self.pool, self.pool8]
        ws = torch.empty(argus.fork_workspace_bytes(self.rows, pools), dtype=torch.uint8, device=DEV)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        argus.fork_pages(self.g, i32(parents), i32(new), W.BF16, pools, self.ref, out, self.codec, self.table, self.lens, c, t, n,
                         MAXP, ws, status=self.status)
        self.table, self.codec, self.lens, self.ref = t, c, n, out
        self.tokens = [(list(self.tokens[p][0]), list(self.tokens[p][1])) if p >= 0 else ([], []) for p in parents]
        self.q_start = i32([0] + np.cumsum(new).tolist())
        self.new = new

    def step(self, seed):
        """New tokens for every row: positions, append, attention; checked against the dense computation."""
        total = sum(self.new)
        qkv = W.normal((total, Hq + 2 * Hkv, D), W.BF16, seed).to(DEV)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        pos = torch.from_numpy(np.random.default_rng(seed).integers(0, 500, (3, total)).astype(np.int32)).to(DEV)
        q_out, out = torch.empty((2, total, Hq, D), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((total, Hq), dtype=torch.float32, device=DEV)
        argus.rope_append(self.g, q, k, v, q_out, self.q_start, self.lens, pos, self.inv, self.pool, self.codec, self.table, MAXP,
                          pair_axis=self.axis, status=self.status)
        args = argus.extend_args(self.g, q_out, self.q_start, [self.pool, self.pool8], self.codec, self.table, self.lens, MAXP,
                                 1.0 / math.sqrt(D), out, lse2_out=lse, status=self.status)
        argus.paged_extend_attn(args, torch.empty(argus.extend_workspace_bytes(args), dtype=torch.uint8, device=DEV))
        torch.cuda.synchronize()
        assert int(self.status) == 0
        # the turned rows, rounded as stored: within half a step of the oracle's
        to64 = lambda x: C.bf16_bits_to_f64(W.to_bits(x.contiguous()))  # noqa: E731
        kr = oracle.rotate(to64(k), pos.cpu().numpy(), self.inv.cpu().numpy(), self.axis.cpu().numpy(), False)
        table, lens = self.table.cpu().numpy(), self.lens.cpu().numpy()
        t = 0
        for b, n in enumerate(self.new):
            for i in range(n):
                at = int(lens[b]) - n + i
                row = to64(self.pool.codes[int(table[b, at // P]), :, :, at % P])
                # half a step, doubled for the oracle's and the kernel's value on two sides of a rounding border
                assert np.abs(row[0] - kr[t]).max() <= 2 * 2.0 ** -8 * np.abs(kr[t]).max()
                assert np.array_equal(row[1], to64(v[t:t + 1])[0])
                self.tokens[b][0].append(row[0])
                self.tokens[b][1].append(row[1])
                t += 1
        self.check(to64(q_out), out, lse)

    def check(self, q, out, lse):
        t = 0
        got = out.float().cpu().numpy()
        for b, n in enumerate(self.new):
            ks, vs = np.array(self.tokens[b][0]), np.array(self.tokens[b][1])
            for i in range(n):
                see = len(ks) - n + i + 1
                for h in range(Hq):
                    s = ks[:see, h // (Hq // Hkv)] @ q[t, h] / math.sqrt(D)
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    ref, av = w @ vs[:see, h // (Hq // Hkv)], w @ np.abs(vs[:see, h // (Hq // Hkv)])
                    # p and the result rounded to bf16 once each; scores of a few units in fp32
                    assert np.all(np.abs(got[t, h] - ref) <= 2.0 ** -8 * (av + np.abs(ref)) + 1e-4 * av + 1e-30)
                    assert abs(float(lse[t, h]) - (s.max() + math.log(np.exp(s - s.max()).sum())) / math.log(2)) <= 1e-4
                t += 1

    def demote_first_pages(self):
        """Page 0 of row 0 to FP8 (it is held by row 0 alone)."""
        slot = int(self.table[0, 0])
        assert int(self.ref[0][slot]) == 1
        dst = int((self.ref[1] == 0).nonzero()[0])
        i32 = lambda x: torch.tensor([x], dtype=torch.int32, device=DEV)  # noqa: E731
        argus.quantize_pages(self.g, W.BF16, self.pool.codes, self.n16, i32(slot), self.pool8, i32(dst), 1)
        self.table[0, 0], self.codec[0, 0] = dst, W.FP8_E4M3
        self.ref[0][slot] -= 1
        self.ref[1][dst] += 1
        codes, meta = self.pool8.codes[dst].cpu(), self.pool8.meta[dst].cpu().double()
        x = codes.view(torch.float8_e4m3fn).double() * meta[:, :, None, None]
        for i in range(P):
            self.tokens[0][0][i], self.tokens[0][1][i] = x[0, :, i].numpy(), x[1, :, i].numpy()

    def compact(self):
        for k, pool in enumerate((self.pool, self.pool8)):
            t, r = torch.empty_like(self.table), torch.empty_like(self.ref[k])
            live = torch.empty(1, dtype=torch.int32, device=DEV)
            ws = torch.empty(argus.compact_workspace_bytes(pool), dtype=torch.uint8, device=DEV)
            argus.compact_pages(self.g, pool, self.ref[k], r, self.codec, self.table, self.lens, t, MAXP, live, ws, status=self.status)
            self.table, self.ref[k] = t, r
            n = int(live)
            assert torch.all(r[:n] > 0) and torch.all(r[n:] == 0)


def test_a_servers_steps():
    s = Server(6, 96)
    s.fork([0, 1, -1, -1, -1, -1], [50, 37, 0, 0, 0, 0])       # two prompts
    s.step(1)
    s.demote_first_pages()
    s.fork([0, 1, 0, 0, 1, -1], [1, 1, 1, 1, 1, 0])            # beams of both
    s.step(2)
    s.fork([2, 2, 3, 0, 1, 1], [1, 3, 1, 20, 1, 1])            # reordered; one row takes a chunk
    s.step(3)
    s.compact()
    s.fork([0, -1, 2, 3, 4, -1], [2, 0, 0, 1, 16, 0])          # two rows freed
    s.step(4)
    s.compact()
    s.fork([0, 1, 2, 3, 4, 5], [1, 5, 1, 1, 1, 19])            # ... which start anew
    s.step(5)
    # the counts are the table's references
    table, codec, lens = s.table.cpu().numpy(), s.codec.cpu().numpy(), s.lens.cpu().numpy()
    for k, c in enumerate((W.BF16, W.FP8_E4M3)):
        held = np.zeros(96, int)
        for b in range(6):
            for j in range((lens[b] + P - 1) // P):
                if codec[b, j] == c:
                    held[table[b, j]] += 1
        assert np.array_equal(held, s.ref[k].cpu().numpy())
