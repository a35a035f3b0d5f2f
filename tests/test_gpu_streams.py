"""Calls that run at the same time on two streams, with outputs and workspaces of their own: the bits of the same calls one
by one.  Every launch of both streams is queued behind one event before the first of them can start."""

import numpy as np
import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus
from mixed_precision_paged_argus_gb300 import workloads as W
import test_gpu_accept
import test_gpu_evict
import test_gpu_rope
from test_gpu_extend import DEV, make
from test_gpu_masks import args_of, tree, words_of

pytestmark = pytest.mark.gpu
ROUNDS = 4


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def window_tree_and_weights(seed):
    c = make(8, 2, 128, 16, [900, 40, 333], [9, 40, 33], [W.BF16, W.FP8_E4M3], W.BF16, seed=seed)
    mask = words_of([tree(n, n) for n in c.new], 2)
    (args, ws, out, lse), (args2, ws2, out2, lse2), (args3, ws3, out3, lse3) = args_of(c), args_of(c), args_of(c)
    w = torch.zeros((3, 2, c.max_pages * 16), device=DEV)

    def launch(stream, _):
        argus.paged_window_extend_attn(args, ws, 100, 4, stream=stream)
        argus.paged_tree_attn(args2, ws2, mask, stream=stream)
        argus.paged_extend_attn(args3, ws3, stream=stream)
        argus.attn_weights(args3, w, 0.5, stream=stream)
    return launch, [out, lse, out2, lse2, out3, lse3, w]


def weights_of_group_codes(seed):
    c = make(8, 2, 128, 16, [1900, 40, 333, 700], [21, 1, 0, 1], [W.BF16, W.INT4_G32], W.BF16, seed=seed)
    lse, w = torch.linspace(7, 9, 23 * 8, device=DEV).view(23, 8), torch.zeros((4, 2, c.max_pages * 16), device=DEV)
    args = argus.extend_args(c.g, c.q, dev(c.q_start), c.pools, c.d_codec, c.d_table, c.d_lens, c.max_pages, c.scale, None, lse2_out=lse)

    def launch(stream, _):
        argus.attn_weights(args, w, 0.5, stream=stream)
    return launch, [w]


def eviction(seed):
    c = make(8, 2, 128, 16, [3000, 40, 1333], [1, 1, 1], [W.BF16, W.FP8_E4M3], W.BF16, seed=seed)
    w, table = dev(test_gpu_evict.weights(c, seed)), torch.arange(39, dtype=torch.int32, device=DEV).view(3, 13).flip(0).contiguous()
    dst = argus.Pool.empty(W.FP8_E4M3, 39, 2, 16, 128, device=DEV, zero=True)
    lens, kept, w_out = (torch.zeros(s, dtype=t, device=DEV) for s, t in ((3, torch.int32), ((3, 2, 200), torch.int32), ((3, 2, 210), torch.float32)))

    def launch(stream, _):
        argus.evict_tokens(c.g, c.pools, c.d_codec, c.d_table, c.d_lens, c.max_pages, w, 200, 4, 50, dst, table, 13, lens, kept, w_out, stream=stream)
    return launch, [dst.codes.view(torch.uint8), dst.meta, lens, kept, w_out]


def norms(seed):
    s = test_gpu_rope.case(14, 2, 64, 16, W.BF16, [5, 100, 0], [300, 1, 77], 64, 2, seed=seed)
    q_out = torch.zeros(s["q"].shape, dtype=s["q"].dtype, device=DEV)
    wq, wk = torch.rand(64, device=DEV, generator=torch.Generator(DEV).manual_seed(seed)), torch.linspace(0.5, 2, 64, device=DEV)
    q_start, pos, inv, axis, codec, table = (dev(s[k]) for k in ("q_start", "pos", "inv", "axis", "codec", "table"))
    lens = torch.tensor(s["lens"], dtype=torch.int32, device=DEV)
    pool = argus.Pool(s["kind"], s["pool"], None, s["n_slots"])

    def launch(stream, _):
        argus.norm_rope_append(s["g"], s["q"], s["k"], s["v"], q_out, q_start, lens, pos, inv, pool, codec, table, s["max_pages"], wq, wk, 1e-6,
                               pair_axis=axis, stream=stream)
    return launch, [q_out, s["pool"]]


def accepted(seed):
    rng = np.random.default_rng(seed)
    new = rng.integers(1, 60, 40).tolist()
    paths = [sorted(rng.choice(n, size=int(rng.integers(0, n + 1)), replace=False).tolist()) for n in new]
    s = test_gpu_accept.case(2, 64, 16, W.FP16, [n + int(rng.integers(0, 200)) for n in new], new, paths, seed=seed)
    pools = [s["pool"].clone() for _ in range(ROUNDS)]   # rows move in place
    codec, table, q_start, lens, path, n_path = (dev(s[k]) for k in ("codec", "table", "q_start", "lens", "path", "n_path"))
    out = torch.zeros(len(new), dtype=torch.int32, device=DEV)

    def launch(stream, i):
        argus.accept_tokens(s["g"], argus.Pool(s["kind"], pools[i], None, s["n_slots"]), codec, table, s["max_pages"], q_start, lens, path, n_path, out,
                            stream=stream)
    return launch, [out, *pools]


def test_every_operator_of_drafts_and_short_caches_on_two_streams_together():
    build = lambda seed: [f(seed) for f in (window_tree_and_weights, weights_of_group_codes, eviction, norms, accepted)]  # noqa: E731
    alone = [build(900), build(901)]
    for calls in alone:
        for i in range(ROUNDS):
            for launch, _ in calls:
                launch(torch.cuda.current_stream(), i)
                torch.cuda.synchronize()
    together = [build(900), build(901)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    begin, end = ([torch.cuda.Event(enable_timing=True) for _ in streams] for _ in range(2))
    busy, gate = torch.empty(2 << 30, dtype=torch.uint8, device=DEV), torch.cuda.Event()
    torch.cuda.synchronize()
    for _ in range(24):                                  # some milliseconds, while the launches are queued
        busy.fill_(1)
    gate.record()
    for s, e in zip(streams, begin):
        s.wait_event(gate)
        e.record(s)
    for i in range(ROUNDS):
        for which in zip(*together):
            for (launch, _), s in zip(which, streams):
                launch(s, i)
    for s, e in zip(streams, end):
        e.record(s)
    queued = not gate.query()
    torch.cuda.synchronize()
    assert queued and begin[1].elapsed_time(end[0]) > 0 and begin[0].elapsed_time(end[1]) > 0
    for calls, others in zip(alone, together):
        for (_, want), (_, got) in zip(calls, others):
            for x, y in zip(want, got):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
