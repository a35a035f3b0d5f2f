"""argus_attn_weights where few sequences have most of the rows: one call's two kernels share the sequences between
them, and what follows waits for both."""

import numpy as np
import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus
from mixed_precision_paged_argus_gb300 import workloads as W
from test_gpu_extend import DEV, F8, I8, make, spoil_tails
from test_gpu_weights import args_of, check

pytestmark = pytest.mark.gpu
SHARES = [(W.BF16, [F8]), (W.BF16, [W.BF16, I8]), (W.FP16, [W.FP16]), (W.BF16, [W.INT4_G32, F8]), (W.FP16, [W.FP16, W.INT2_G32])]


@pytest.mark.parametrize("dtype,codecs", SHARES)
@pytest.mark.parametrize("new", [[33] + [0] * 30, [0] * 15 + [21] + [0] * 15, [2, 0, 3] * 5, [40, 1, 0, 1, 5] + [1] * 15, [1] * 16, [16] + [0] * 15, [5, 4] * 8])
def test_idle_slots_and_long_questions(new, dtype, codecs):
    c = make(8, 2, 128, 16, [(700, 40, 0, 65, 233)[b % 5] + n for b, n in enumerate(new)], new, codecs, dtype, seed=700 + len(new))
    if all(k <= I8 for k in codecs):
        spoil_tails(c)
    check(c, decay=0.5)
    check(c, causal=False, decay=0.0)


def case(seed, dtype, codecs, new):
    c = make(16, 2, 128, 16, [9000] + [1500 + 100 * b for b in range(len(new) - 1)], new, codecs, dtype, seed=seed)
    lse = 8 + torch.rand((int(c.q_start[-1]), 16), device=DEV, generator=torch.Generator(DEV).manual_seed(seed))
    return c, args_of(c, lse), torch.zeros((len(new), 2, c.max_pages * 16), device=DEV)


@pytest.mark.parametrize("dtype,codecs", [SHARES[0], SHARES[1], SHARES[3]])
def test_what_follows_waits_for_both_kernels(dtype, codecs):
    """Calls on the same weights right behind each other, with a copy behind each, in a graph: the bits of calls one by one."""
    for new in ([64] + [1] * 20, [2] + [3] * 20, [100] + [0] * 20):
        _, args, w = case(800, dtype, codecs, new)
        want = []
        for _ in range(4):
            torch.cuda.synchronize()
            argus.attn_weights(args, w, 0.75)
            torch.cuda.synchronize()
            want.append(w.clone())
        got = [torch.empty_like(w) for _ in want]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w.zero_()
            for x in got:
                argus.attn_weights(args, w, 0.75)
                x.copy_(w)
        for _ in range(3):
            for x in got:
                x.fill_(-1)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_replayed_with_other_shares():
    """One graph, other token counts: a sequence changes from one kernel to the other."""
    for dtype, codecs in (SHARES[0], SHARES[3]):
        c, args, w = case(810, dtype, codecs, [30, 1, 1, 1, 7])
        q_start = args._keep[3]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            argus.attn_weights(args, w, 0.0)
        for new in ([1, 30, 1, 1, 7], [8, 8, 8, 8, 8], [0, 0, 0, 0, 40], [30, 1, 1, 1, 7]):
            q_start.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)))
            graph.replay()
            got = w.clone()
            w.fill_(-1)
            argus.attn_weights(args, w, 0.0)
            for b, n in enumerate(c.lens):
                assert torch.equal(got[b, :, :int(n)], w[b, :, :int(n)])
