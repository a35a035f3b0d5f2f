"""The operators of a paged cache's life, measured: their plain forms and the library's calls.

  extend   several query tokens per sequence (a ragged batch) attend to the paged cache, whose pages
           are 16-bit, FP8 or INT8 with one scale per page, KV head and K|V; causal over a sequence's
           own cache, or full over an encoder's states of another length (cross attention)
  rope     rotary positions with one or several axes on the new tokens' q and k, and the append of
           k and v to the sequences' 16-bit pages
  fork     one step of a cache's page table: rows forked from their parents, rows freed, shared
           partial pages copied before they are appended to, pages allocated for the new tokens
  compact  the live pages of a pool moved into its lowest slots, the block table rewritten

With `own` false, `run` computes each in elementary torch operations; with `own` true it makes the
library's calls.  The lengths of a case follow from the case alone, its values from the seed.
"""

import math
import random

import numpy as np
import torch

own = False

FP16, BF16, FP8, INT8 = 0, 1, 2, 3
KINDS = {"fp16": (FP16, torch.float16), "bf16": (BF16, torch.bfloat16)}
LOG2E = 1.0 / math.log(2.0)


# ---------------------------------------------------------------- cases

def _extend(name, batch, hq, hkv, d, page, dtype, cache, len_lo, len_hi, nq_lo, nq_hi, causal):
    c = dict(op="extend", batch=batch, hq=hq, hkv=hkv, d=d, page=page, dtype=dtype, cache=cache,
             len_lo=len_lo, len_hi=len_hi, nq_lo=nq_lo, nq_hi=nq_hi, causal=causal)
    return dict(c, name=name) if name else c


def _rope(name, batch, hq, hkv, d, page, dtype, rot, axes, adjacent, cached, new_lo, new_hi):
    c = dict(op="rope", batch=batch, hq=hq, hkv=hkv, d=d, page=page, dtype=dtype, rot=rot, axes=axes,
             adjacent=adjacent, cached=cached, new_lo=new_lo, new_hi=new_hi)
    return dict(c, name=name) if name else c


def _fork(name, batch, hkv, d, page, dtype, len_lo, len_hi, spare, change, new_hi):
    c = dict(op="fork", batch=batch, hkv=hkv, d=d, page=page, dtype=dtype, len_lo=len_lo, len_hi=len_hi,
             spare=spare, change=change, new_hi=new_hi)
    return dict(c, name=name) if name else c


def _compact(name, batch, hkv, d, page, dtype, slots, live):
    c = dict(op="compact", batch=batch, hkv=hkv, d=d, page=page, dtype=dtype, slots=slots, live=live)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a few drafted tokens of one small model's sequence are verified at once: latency counts
        _extend("verify-one", 1, 14, 2, 64, 1024, "fp16", "16", 4096, 4096, 4, 4, True),
        # drafted tokens of a serving batch, FP8 pages of 16 tokens, long ragged contexts: bytes count
        _extend("verify-batch-fp8", 32, 32, 8, 128, 16, "bf16", "fp8", 8192, 32768, 1, 8, True),
        # a step that mixes single tokens and prompt chunks over three tiers
        _extend("mixed-tiers", 8, 32, 4, 128, 64, "bf16", "mixed", 500, 16384, 1, 256, True),
        # a decoder's prompts read an encoder's states held in INT8 (an audio or image encoder's length)
        _extend("cross-int8", 16, 16, 2, 128, 16, "fp16", "int8", 1, 1500, 1, 256, False),
        # one chunk of a long prompt over its own FP8 cache: arithmetic counts
        _extend("chunk-long-fp8", 1, 16, 2, 128, 64, "bf16", "fp8", 131072, 131072, 1024, 1024, True),
        # the positions and the append of one decode step of a serving batch
        _rope("append-step", 32, 32, 8, 128, 16, "bf16", 128, 3, False, 32768, 1, 1),
        # prompt chunks of several sequences, odd lengths
        _rope("append-prompts", 5, 32, 8, 128, 16, "bf16", 128, 3, False, 1001, 777, 2048),
        # a video's tokens of a small model: adjacent pairs, part of the head rotated
        _rope("append-video", 2, 14, 2, 64, 1024, "fp16", 32, 3, True, 0, 20000, 32768),
        # a beam step of one small request: latency counts
        _fork("beams-small", 8, 2, 64, 64, "fp16", 100, 1000, 64, 0.75, 1),
        # a scheduler's step for a large batch: some rows forked, some freed, all appended to
        _fork("fork-batch", 512, 8, 128, 16, "bf16", 1, 8192, 8192, 0.25, 40),
        # a small pool with a few holes
        _compact("compact-small", 4, 2, 64, 64, "fp16", 96, 0.6),
        # a large pool shrunk to give memory back
        _compact("compact-large", 64, 8, 128, 16, "bf16", 16384, 0.5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["extend", "extend", "extend", "rope", "fork", "compact"])
    hq, hkv, d, page = rng.choice([(14, 2, 64, 1024), (32, 8, 128, 16), (32, 4, 128, 64), (16, 2, 128, 64), (6, 6, 64, 48)])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "extend":
        batch = _log(rng, 1, 24)
        hi = _log(rng, 64, min(32768, 200000 // batch))
        nq = _log(rng, 1, 300)
        return _extend(None, batch, hq, hkv, d, page, dtype, rng.choice(["16", "fp8", "int8", "mixed"]),
                       rng.randint(0, hi), hi, rng.randint(1, nq), nq, rng.random() < 0.7)
    if op == "rope":
        hi = _log(rng, 1, 5000)
        return _rope(None, _log(rng, 1, 8), hq, hkv, d, page, dtype, rng.choice([16, 32, d]), rng.choice([1, 2, 3]),
                     rng.random() < 0.5, _log(rng, 1, 30000), rng.randint(1, hi), hi)
    if op == "fork":
        batch = _log(rng, 1, 300)
        hi = _log(rng, page, 8192)
        return _fork(None, batch, hkv, d, page, dtype, rng.randint(0, hi), hi, _log(rng, 8, 4096) + 2 * batch,
                     rng.choice([0.1, 0.4, 0.8]), rng.randint(0, 70))
    return _compact(None, _log(rng, 1, 100), hkv, d, page, dtype,
                    _log(rng, 16, min(12000, (1 << 30) // (4 * hkv * page * d))), rng.choice([0.1, 0.4, 0.7, 0.95]))


def _rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """Per-sequence lengths and new tokens: the first sequences take the ends of the ranges."""
    r, n = _rng(case), case["batch"]
    lens = [case["len_hi"], case["len_lo"]][:n] + [r.randint(case["len_lo"], case["len_hi"]) for _ in range(n - 2)]
    new = [case["nq_hi"], case["nq_lo"]][:n] + [r.randint(case["nq_lo"], case["nq_hi"]) for _ in range(n - 2)]
    if case["causal"]:   # the cache already holds the new tokens
        lens = [max(a, b) for a, b in zip(lens, new)]
    return lens, new


def _ceil(a, b):
    return (a + b - 1) // b


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(new):
    return _ints([0] + np.cumsum(new).tolist())


def prepare(case, seed):
    return {"extend": _prepare_extend, "rope": _prepare_rope, "fork": _prepare_fork, "compact": _prepare_compact}[case["op"]](case, seed)


def _prepare_extend(case, seed):
    g = _gen(seed)
    kind, dtype = KINDS[case["dtype"]]
    lens, new = _lengths(case)
    b, p, hkv, d = case["batch"], case["page"], case["hkv"], case["d"]
    max_pages = max(1, _ceil(max(lens), p))
    n_pages = np.array([_ceil(n, p) for n in lens])
    logical = np.arange(max_pages)[None, :]
    used = logical < n_pages[:, None]
    age = n_pages[:, None] - 1 - logical          # 0: the newest page
    codec = {"16": np.full(used.shape, kind), "fp8": np.full(used.shape, FP8), "int8": np.full(used.shape, INT8),
             "mixed": np.where(age < 4, kind, np.where(age < n_pages[:, None] // 2, FP8, INT8))}[case["cache"]]
    codec = np.where(used, codec, 0)
    table = np.zeros(used.shape, np.int64)
    perm = np.random.default_rng(int(seed))
    pools = {}
    for c in (kind, FP8, INT8):
        n = int((used & (codec == c)).sum())
        if n == 0:
            continue
        table[used & (codec == c)] = perm.permutation(n)
        shape = (n, 2, hkv, p, d)
        if c == kind:
            pools[c] = (_randn(shape, dtype, g), None)
        elif c == FP8:
            x = torch.randn(shape, generator=g, device="cuda") * 100.0
            codes = x.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
            pools[c] = (codes, 0.008 + 0.004 * torch.rand((n, 2, hkv), generator=g, device="cuda"))
        else:
            x = torch.randn(shape, generator=g, device="cuda") * 30.0
            codes = x.round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
            pools[c] = (codes, 0.025 + 0.015 * torch.rand((n, 2, hkv), generator=g, device="cuda"))
    return dict(case=case, kind=kind, dtype=dtype, max_pages=max_pages, nq_max=max(new),
                q=_randn((sum(new), case["hq"], d), dtype, g), q_start=_starts(new), seq_lens=_ints(lens), pools=pools,
                page_codec=torch.from_numpy(codec.astype(np.uint8)).cuda(), block_table=torch.from_numpy(table.astype(np.int32)).cuda(),
                scale=1.0 / math.sqrt(d))


def _rope_lengths(case):
    r, n = _rng(case), case["batch"]
    new = [case["new_hi"], case["new_lo"]][:n] + [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n - 2)]
    return [r.randint(case["cached"] // 2, case["cached"]) for _ in range(n)], new


def _prepare_rope(case, seed):
    g = _gen(seed)
    kind, dtype = KINDS[case["dtype"]]
    cached, new = _rope_lengths(case)
    b, p, hq, hkv, d, rot, axes = (case[k] for k in ("batch", "page", "hq", "hkv", "d", "rot", "axes"))
    total = sum(new)
    qkv = _randn((total, (hq + 2 * hkv) * d), dtype, g)      # a fused projection's rows
    lens = [a + n for a, n in zip(cached, new)]
    max_pages = _ceil(max(lens), p)
    first = [a // p for a in cached]
    last = [_ceil(n, p) for n in lens]
    n_slots = sum(l - f for f, l in zip(first, last))        # the pages written; older ones lie elsewhere
    table = np.full((b, max_pages), 0, np.int32)
    perm, k = np.random.default_rng(int(seed)).permutation(n_slots), 0
    for i in range(b):
        table[i, first[i]:last[i]] = perm[k:k + last[i] - first[i]]
        k += last[i] - first[i]
    # positions of time, height and width: text counts up, frames hold still in time
    at = torch.cat([torch.arange(a, a + n, device="cuda") for a, n in zip(cached, new)])
    noise = torch.randint(0, 64, (3, total), generator=g, device="cuda")
    pos = torch.stack([at, at // 7 + noise[1], at // 11 + noise[2]])[:axes].to(torch.int32).contiguous()
    half = rot // 2
    inv_freq = torch.tensor([10000.0 ** (-i / half) for i in range(half)], dtype=torch.float64, device="cuda")
    pair_axis = torch.arange(half, device="cuda").mul(axes).div(half, rounding_mode="floor").to(torch.uint8)
    return dict(case=case, kind=kind, dtype=dtype, max_pages=max_pages, q=qkv[:, :hq * d].view(total, hq, d),
                k=qkv[:, hq * d:(hq + hkv) * d].view(total, hkv, d), v=qkv[:, (hq + hkv) * d:].view(total, hkv, d),
                q_start=_starts(new), seq_lens=_ints(lens), positions=pos, inv_freq=inv_freq, pair_axis=pair_axis,
                pool=_randn((n_slots, 2, hkv, p, d), dtype, g), page_codec=torch.full((b, max_pages), kind, dtype=torch.uint8, device="cuda"),
                block_table=torch.from_numpy(table).cuda())


def _fork_lengths(case):
    r, n = _rng(case), case["batch"]
    lens = [case["len_hi"], case["len_lo"]][:n] + [r.randint(case["len_lo"], case["len_hi"]) for _ in range(n - 2)]
    parents = []
    for i in range(n):
        x = r.random()
        parents.append(i if x >= case["change"] else -1 if x < 0.2 * case["change"] else r.randrange(n))
    new = [r.randint(0, case["new_hi"]) for _ in range(n)]
    return lens, parents, new


def _fork_sizes(case):
    lens, parents, new = _fork_lengths(case)
    p = case["page"]
    max_pages = max(1, _ceil(max(lens) + case["new_hi"], p))
    newest = [_ceil(n, p) - max(0, _ceil(n, p) - 4) for n in lens]     # the newest 4 pages are 16-bit
    older = [_ceil(n, p) - k for n, k in zip(lens, newest)]
    return lens, parents, new, max_pages, newest, older


def _prepare_fork(case, seed):
    g = _gen(seed)
    kind, dtype = KINDS[case["dtype"]]
    b, p, hkv, d = case["batch"], case["page"], case["hkv"], case["d"]
    lens, parents, new, max_pages, newest, older = _fork_sizes(case)
    logical = np.arange(max_pages)[None, :]
    old = logical < np.array(older)[:, None]
    recent = ~old & (logical < (np.array(older) + np.array(newest))[:, None])
    n16, n8 = sum(newest) + case["spare"], max(1, sum(older))
    perm = np.random.default_rng(int(seed))
    table = np.full((b, max_pages), -1, np.int32)
    slots16 = perm.permutation(n16)[:sum(newest)]
    table[recent] = slots16
    table[old] = perm.permutation(n8)[:sum(older)]
    codec = np.where(old, FP8, np.where(recent, kind, 0)).astype(np.uint8)
    ref16 = np.zeros(n16, np.int32)
    ref16[slots16] = 1
    # a few slots are held by a prefix cache as well: tails among them may not be written in place
    ref16[slots16[::5]] += 1
    ref8 = np.zeros(n8, np.int32)
    ref8[table[old]] = 1
    cu = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    return dict(case=case, kind=kind, dtype=dtype, max_pages=max_pages, pool=_randn((n16, 2, hkv, p, d), dtype, g),
                pool8=torch.zeros((n8, 2, hkv, p, d), dtype=torch.uint8, device="cuda"), meta8=torch.ones((n8, 2, hkv), device="cuda"),
                ref16=cu(ref16), ref8=cu(ref8), block_table=cu(table), page_codec=cu(codec), seq_lens=_ints(lens),
                parents=_ints(parents), n_new=_ints(new))


def _compact_sizes(case):
    r = _rng(case)
    lens = [0] * case["batch"]
    live = max(1, min(case["slots"], int(case["live"] * case["slots"])))
    for _ in range(live):
        lens[r.randrange(case["batch"])] += case["page"]
    lens = [max(0, n - r.randrange(case["page"])) if n else 0 for n in lens]
    return lens, max(1, max(_ceil(n, case["page"]) for n in lens))


def _prepare_compact(case, seed):
    g = _gen(seed)
    kind, dtype = KINDS[case["dtype"]]
    b, p = case["batch"], case["page"]
    lens, max_pages = _compact_sizes(case)
    used = np.arange(max_pages)[None, :] < np.array([_ceil(n, p) for n in lens])[:, None]
    table = np.full((b, max_pages), -1, np.int32)
    # live pages lie anywhere in the pool: the seed says where
    slots = np.random.default_rng(int(seed)).permutation(case["slots"])[:int(used.sum())]
    table[used] = slots
    ref = np.zeros(case["slots"], np.int32)
    ref[slots] = 1
    cu = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    return dict(case=case, kind=kind, dtype=dtype, max_pages=max_pages, pool=_randn((case["slots"], 2, case["hkv"], p, case["d"]), dtype, g),
                ref=cu(ref), block_table=cu(table), page_codec=torch.full((b, max_pages), kind, dtype=torch.uint8, device="cuda"),
                seq_lens=_ints(lens))


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"extend": _own_extend, "rope": _own_rope, "fork": _own_fork, "compact": _own_compact}[op](state)
    return {"extend": _plain_extend, "rope": _plain_rope, "fork": _plain_fork, "compact": _plain_compact}[op](state)


def _argus():
    import mixed_precision_paged_argus_gb300.argus as argus
    return argus


def _geom(argus, c):
    return argus.geom(c.get("hq", c["hkv"]), c["hkv"], c["d"], c["page"])


def _own_extend(s):
    argus, c = _argus(), s["case"]
    pools = [argus.Pool(k, codes, meta, codes.shape[0]) for k, (codes, meta) in s["pools"].items()]
    out = torch.empty(s["q"].shape, dtype=s["dtype"], device="cuda")
    lse2 = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    args = argus.extend_args(_geom(argus, c), s["q"], s["q_start"], pools, s["page_codec"], s["block_table"], s["seq_lens"],
                             s["max_pages"], s["scale"], out, causal=c["causal"], lse2_out=lse2)
    ws = torch.empty(argus.extend_workspace_bytes(args), dtype=torch.uint8, device="cuda")
    argus.paged_extend_attn(args, ws)
    return out, lse2


def _own_rope(s):
    argus, c = _argus(), s["case"]
    q_out = torch.empty(s["q"].shape, dtype=s["dtype"], device="cuda")
    pool = argus.Pool(s["kind"], s["pool"], None, s["pool"].shape[0])
    argus.rope_append(_geom(argus, c), s["q"], s["k"], s["v"], q_out, s["q_start"], s["seq_lens"], s["positions"], s["inv_freq"],
                      pool, s["page_codec"], s["block_table"], s["max_pages"], pair_axis=s["pair_axis"], adjacent=c["adjacent"])
    return q_out, s["pool"]


def _own_fork(s):
    argus, c = _argus(), s["case"]
    pools = [argus.Pool(s["kind"], s["pool"], None, s["pool"].shape[0]), argus.Pool(FP8, s["pool8"], s["meta8"], s["pool8"].shape[0])]
    table, codec = torch.empty_like(s["block_table"]), torch.empty_like(s["page_codec"])
    lens, ref16, ref8 = torch.empty_like(s["seq_lens"]), torch.empty_like(s["ref16"]), torch.empty_like(s["ref8"])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = _geom(argus, c)
    ws = torch.empty(argus.fork_workspace_bytes(c["batch"], pools), dtype=torch.uint8, device="cuda")
    argus.fork_pages(g, s["parents"], s["n_new"], s["kind"], pools, [s["ref16"], s["ref8"]], [ref16, ref8], s["page_codec"],
                     s["block_table"], s["seq_lens"], codec, table, lens, s["max_pages"], ws, status=status)
    return table, codec, lens, ref16, ref8, s["pool"], status


def _own_compact(s):
    argus, c = _argus(), s["case"]
    pool = argus.Pool(s["kind"], s["pool"], None, s["pool"].shape[0])
    table, ref = torch.empty_like(s["block_table"]), torch.empty_like(s["ref"])
    n_live = torch.empty(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(argus.compact_workspace_bytes(pool), dtype=torch.uint8, device="cuda")
    argus.compact_pages(_geom(argus, c), pool, s["ref"], ref, s["page_codec"], s["block_table"], s["seq_lens"], table,
                        s["max_pages"], n_live, ws)
    return table, ref, s["pool"], n_live


# ---- extend, plainly: the pages' values gathered in 32 bits, padded scores, masked softmax

def _values(codec, codes, meta):
    if codec == FP8:
        return codes.view(torch.float8_e4m3fn).float() * meta[..., None, None]
    if codec == INT8:
        return codes.view(torch.int8).float() * meta[..., None, None]
    return codes.float()


def _fill(pages, s, codec):
    """The pages of one codec, dequantised, at their places in [B, max_pages, 2, Hkv, P, D]."""
    if codec in s["pools"]:
        at = torch.arange(s["max_pages"], device="cuda")[None, :] < (s["seq_lens"][:, None] + s["case"]["page"] - 1) // s["case"]["page"]
        at = at & (s["page_codec"] == codec)
        slots = s["block_table"][at].long()
        codes, meta = s["pools"][codec]
        pages[at] = _values(codec, codes[slots], None if meta is None else meta[slots])


def _plain_extend(s):
    c = s["case"]
    b, hq, hkv, d, p, mp, nq = c["batch"], c["hq"], c["hkv"], c["d"], c["page"], s["max_pages"], s["nq_max"]
    grp = hq // hkv
    pages = torch.zeros((b, mp, 2, hkv, p, d), dtype=torch.float32, device="cuda")
    _fill(pages, s, s["kind"])
    _fill(pages, s, FP8)
    _fill(pages, s, INT8)
    kv = pages.permute(2, 0, 3, 1, 4, 5).reshape(2, b, hkv, mp * p, d)
    del pages
    first, n = s["q_start"][:-1].long(), (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(nq, device="cuda")
    rows = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)                       # [B, nq]
    q = s["q"][rows].float().view(b, nq, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, nq * grp, d)
    scores = torch.matmul(q, kv[0].transpose(2, 3)).mul_(s["scale"]).view(b, hkv, nq, grp, mp * p)
    key = torch.arange(mp * p, device="cuda")
    limit = s["seq_lens"].long()[:, None].expand(b, nq)
    if c["causal"]:
        limit = s["seq_lens"].long()[:, None] - n[:, None] + i + 1
    limit = torch.minimum(limit, s["seq_lens"].long()[:, None])
    scores.masked_fill_((key >= limit[..., None])[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = scores.sum(-1, keepdim=True)
    o = torch.matmul(scores.view(b, hkv, nq * grp, mp * p), kv[1]).view(b, hkv, nq, grp, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse2 = ((top + total.log()) * LOG2E).squeeze(-1)
    real = i < n[:, None]                                                            # padded rows fall away
    out = o.permute(0, 2, 1, 3, 4).reshape(b, nq, hq, d)[real]
    return out.to(s["dtype"]), lse2.permute(0, 2, 1, 3).reshape(b, nq, hq)[real]


# ---- rope, plainly: the angles in 64 bits (far positions), the rotation in 32

def _turned(x, cos, sin, rot, adjacent):
    x = x.float()
    if adjacent:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"][s["pair_axis"].long()].t().double() * s["inv_freq"]        # [T, rot/2]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q_out = _turned(s["q"], cos, sin, c["rot"], c["adjacent"]).to(s["dtype"])
    k = _turned(s["k"], cos, sin, c["rot"], c["adjacent"]).to(s["dtype"])
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    row = torch.repeat_interleave(torch.arange(c["batch"], device="cuda"), n, output_size=s["q"].shape[0])
    at = (s["seq_lens"].long() - n)[row] + torch.arange(s["q"].shape[0], device="cuda") - s["q_start"].long()[row]
    slot = s["block_table"][row, at // c["page"]].long()
    s["pool"][slot, 0, :, at % c["page"]] = k
    s["pool"][slot, 1, :, at % c["page"]] = s["v"]
    return q_out, s["pool"]


# ---- fork, plainly

def _counts(slots, n):
    return torch.zeros(n, dtype=torch.int64, device="cuda").index_add_(0, slots, torch.ones_like(slots))


def _plain_fork(s):
    c = s["case"]
    b, p, mp = c["batch"], c["page"], s["max_pages"]
    logical = torch.arange(mp, device="cuda")[None, :]
    par = s["parents"].long()
    kept = torch.where(par >= 0, s["seq_lens"].long()[par.clamp(min=0)], 0)
    table, codec = s["block_table"].long()[par.clamp(min=0)], s["page_codec"].long()[par.clamp(min=0)]
    pages = (kept + p - 1) // p
    before = logical < ((s["seq_lens"].long() + p - 1) // p)[:, None]
    now = logical < pages[:, None]
    refs = {}
    for name, k in (("ref16", s["kind"]), ("ref8", FP8)):
        n = s[name].shape[0]
        refs[name] = s[name].long() - _counts(s["block_table"].long()[before & (s["page_codec"] == k)], n) + _counts(table[now & (codec == k)], n)
    ref16 = refs["ref16"]
    new = torch.where(par >= 0, s["n_new"].long(), 0)
    # a partial page that the row appends to is copied unless the row alone holds it; of rows that share
    # one with nobody else, the first keeps it
    row = torch.arange(b, device="cuda")
    tail = (pages - 1).clamp(min=0)
    writes = (kept % p != 0) & (new > 0)
    src = torch.where(writes, table[row, tail], 0)
    n16 = ref16.shape[0]
    writers = torch.zeros(n16, dtype=torch.int64, device="cuda").index_add_(0, src, writes.long())
    lowest = torch.full((n16,), b, dtype=torch.int64, device="cuda").scatter_reduce_(0, src, torch.where(writes, row, b), "amin")
    copied = writes & ~((ref16[src] == writers[src]) & (lowest[src] == row))
    ends = (kept + new + p - 1) // p
    wanted = copied.long() + ends - pages
    first = wanted.cumsum(0) - wanted
    free = torch.nonzero(ref16 == 0).squeeze(1)
    asks = (copied[:, None] & (logical == tail[:, None])) | ((logical >= pages[:, None]) & (logical < ends[:, None]))
    rank = first[:, None] + logical - pages[:, None] + copied.long()[:, None]
    got = asks & (rank < free.shape[0])
    slots = torch.cat([free, free.new_zeros(1)])[rank.clamp(0, free.shape[0])]
    table = torch.where(got, slots, torch.where(asks | ~now, -1, table))
    codec = torch.where(asks, s["kind"], torch.where(now, codec, 0))
    ref16 = ref16.index_add(0, src, -copied.long())
    ref16[slots[got]] = 1
    moved = copied & got[row, tail]
    s["pool"][table[row, tail][moved]] = s["pool"][src[moved]]
    status = (asks & ~got).sum().reshape(1)
    i32 = torch.int32
    return table.to(i32), codec.to(torch.uint8), (kept + new).to(i32), ref16.to(i32), refs["ref8"].to(i32), s["pool"], status.to(i32)


# ---- compact, plainly

def _plain_compact(s):
    c = s["case"]
    live = s["ref"] > 0
    n_live = live.sum()
    slot = torch.arange(live.shape[0], device="cuda")
    src = torch.nonzero(live & (slot >= n_live)).squeeze(1)
    dst = torch.nonzero(~live & (slot < n_live)).squeeze(1)
    s["pool"][dst] = s["pool"][src]
    to = slot.clone()
    to[src] = dst
    ref = torch.where(slot < n_live, s["ref"], 0)
    ref[dst] = s["ref"][src]
    used = torch.arange(s["max_pages"], device="cuda")[None, :] < ((s["seq_lens"] + c["page"] - 1) // c["page"])[:, None]
    moves = used & (s["page_codec"] == s["kind"])
    table = torch.where(moves, to[s["block_table"].long().clamp(min=0)].to(torch.int32), s["block_table"])
    return table, ref, s["pool"], n_live.reshape(1).to(torch.int32)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "extend":
        lens, new = _lengths(c)
        pairs = sum(n * m - (m * (m - 1) // 2 if c["causal"] else 0) for n, m in zip(lens, new))
        tokens, total, p = sum(lens), sum(new), c["page"]
        per = {"16": 2.0, "fp8": 1.0, "int8": 1.0}.get(c["cache"])
        if per is None:
            recent = sum(min(n, 4 * p) for n in lens)
            per = 1.0 + recent / max(1, tokens)
        return {"bytes": 2 * c["hkv"] * c["d"] * per * tokens + total * c["hq"] * (4 * c["d"] + 4), "flops": 4.0 * c["hq"] * c["d"] * pairs}
    if c["op"] == "rope":
        total = sum(_rope_lengths(c)[1])
        return {"bytes": total * (4.0 * (c["hq"] + 2 * c["hkv"]) * c["d"] + 4 * c["axes"]), "flops": 3.0 * total * (c["hq"] + c["hkv"]) * c["rot"]}
    page = 4.0 * c["hkv"] * c["page"] * c["d"]
    if c["op"] == "fork":
        lens, parents, new, max_pages, newest, older = _fork_sizes(c)
        copies = sum(1 for q, n in zip(range(c["batch"]), new) if parents[q] not in (q, -1) and n and lens[parents[q]] % c["page"])
        slots = sum(newest) + c["spare"] + sum(older)
        return {"bytes": 2 * copies * page + 8.0 * slots + 10.0 * c["batch"] * max_pages, "flops": 0}
    lens, max_pages = _compact_sizes(c)
    live = sum(_ceil(n, c["page"]) for n in lens)
    moves = live * (1 - live / c["slots"])       # live pages above the boundary, on average
    return {"bytes": 2 * moves * page + 8.0 * c["slots"] + 8.0 * c["batch"] * max_pages, "flops": 0}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    return {"extend": _exact_extend, "rope": _exact_rope, "fork": _exact_fork, "compact": _exact_compact}[case["op"]](case, seed)


def _exact_extend(case, seed):
    """One sequence and KV head at a time, some rows at a time: o = sum_j w_j v_j / sum_j w_j, w_j = e^(scale q.k_j)."""
    s, c = prepare(case, seed), case
    lens, new = _lengths(case)
    p, grp, f64 = c["page"], c["hq"] // c["hkv"], torch.float64
    out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
    lse2 = torch.full(s["q"].shape[:2], -math.inf, dtype=f64, device="cuda")
    t0 = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        n_pages = _ceil(n, p)
        tiers, slots = s["page_codec"][b, :n_pages].tolist(), s["block_table"][b, :n_pages].long()
        for h in range(c["hkv"] if n else 0):
            kv = torch.empty((2, n_pages, p, c["d"]), dtype=f64, device="cuda")
            for k, (codes, meta) in s["pools"].items():
                at = torch.tensor([i for i, t in enumerate(tiers) if t == k], dtype=torch.long, device="cuda")
                x = codes[slots[at], :, h]
                x = x.view({FP8: torch.float8_e4m3fn, INT8: torch.int8}.get(k, x.dtype)).to(f64)
                if meta is not None:
                    x = x * meta[slots[at], :, h].to(f64)[:, :, None, None]
                kv[:, at] = x.transpose(0, 1)
            keys, vals = kv.view(2, -1, c["d"])[:, :n]
            step = max(1, (1 << 27) // (n * grp))
            for r in range(0, m, step):
                rows = torch.arange(t0 + r, t0 + min(m, r + step), device="cuda")
                q = s["q"][rows, h * grp:(h + 1) * grp].to(f64)
                x = torch.einsum("tgd,nd->tgn", q, keys) * s["scale"]
                if c["causal"]:
                    last = n - m + (rows - t0)
                    x[(torch.arange(n, device="cuda") > last[:, None])[:, None].expand_as(x)] = -math.inf
                lse = torch.logsumexp(x, -1)
                out[rows, h * grp:(h + 1) * grp] = torch.einsum("tgn,nd->tgd", torch.exp(x - lse[..., None]), vals)
                lse2[rows, h * grp:(h + 1) * grp] = lse / math.log(2.0)
        t0 += m
    return out, lse2


def _exact_rope(case, seed):
    s, c = prepare(case, seed), case
    cached, new = _rope_lengths(case)
    rot, half, d = c["rot"], c["rot"] // 2, c["d"]
    i = torch.arange(half, device="cuda")
    one, two = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + half)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[s["pair_axis"].long()].t() * s["inv_freq"])

    def rotate(x):
        y = x.double().clone()
        z = torch.complex(y[..., one], y[..., two]) * turn[:, None]
        y[..., one], y[..., two] = z.real, z.imag
        return y

    pool, k, t = s["pool"].double(), rotate(s["k"]), 0
    for b, (a, n) in enumerate(zip(cached, new)):
        for page in range(a // c["page"], _ceil(a + n, c["page"])):
            lo, hi = max(a, page * c["page"]), min(a + n, (page + 1) * c["page"])
            rows = slice(lo - page * c["page"], hi - page * c["page"])
            slot = int(s["block_table"][b, page])
            pool[slot, 0, :, rows] = k[t + lo - a:t + hi - a].transpose(0, 1)
            pool[slot, 1, :, rows] = s["v"][t + lo - a:t + hi - a].double().transpose(0, 1)
        t += n
    return rotate(s["q"]), pool


def _exact_fork(case, seed):
    """Row after row on the host; the pages' values in 64 bits."""
    s, c = prepare(case, seed), case
    lens, parents, new, max_pages, _, _ = _fork_sizes(case)
    p = c["page"]
    table, codec = s["block_table"].cpu().numpy(), s["page_codec"].cpu().numpy()
    refs = {s["kind"]: s["ref16"].cpu().numpy().copy(), FP8: s["ref8"].cpu().numpy().copy()}
    rows = [[(int(codec[b, j]), int(table[b, j])) for j in range(_ceil(lens[b], p))] for b in range(c["batch"])]
    out = [list(rows[q]) if q >= 0 else [] for q in parents]
    held = [lens[q] if q >= 0 else 0 for q in parents]
    for b, q in enumerate(parents):
        if q != b:
            for k, slot in rows[b]:
                refs[k][slot] -= 1
            for k, slot in out[b]:
                refs[k][slot] += 1
    ref = refs[s["kind"]]
    free = [int(x) for x in np.flatnonzero(ref == 0)]
    writers = {}
    for b in range(c["batch"]):
        if parents[b] >= 0 and new[b] and held[b] % p:
            writers.setdefault(out[b][-1][1], []).append(b)
    keeps = {w[0] for slot, w in writers.items() if ref[slot] == len(w)}
    copies, short = [], 0
    at = 0
    for b in range(c["batch"]):
        if parents[b] < 0:
            continue
        asks = []
        if new[b] and held[b] % p and b not in keeps:
            asks.append(len(out[b]) - 1)
        have = len(out[b])
        out[b] += [None] * (_ceil(held[b] + new[b], p) - have)
        asks += range(have, len(out[b]))
        for j in asks:
            slot = free[at] if at < len(free) else -1
            at += 1
            short += slot < 0
            if j < have:
                ref[out[b][j][1]] -= 1
                if slot >= 0:
                    copies.append((out[b][j][1], slot))
            out[b][j] = (s["kind"], slot)
            if slot >= 0:
                ref[slot] = 1
        held[b] += new[b]
    t = np.full(table.shape, -1, np.int32)
    k = np.zeros(codec.shape, np.uint8)
    for b, row in enumerate(out):
        t[b, :len(row)] = [x[1] for x in row]
        k[b, :len(row)] = [x[0] for x in row]
    pool = s["pool"].double()
    if copies:
        a, z = np.array(copies).T
        pool[torch.from_numpy(z.copy()).cuda()] = s["pool"].double()[torch.from_numpy(a.copy()).cuda()]
    return t, k, np.array(held, np.int32), ref, refs[FP8], pool, np.array([short], np.int32)


def _exact_compact(case, seed):
    s, c = prepare(case, seed), case
    ref = s["ref"].cpu().numpy()
    live = np.flatnonzero(ref)
    src = [int(x) for x in live if x >= len(live)]
    dst = [x for x in range(len(live)) if ref[x] == 0]
    to = dict(zip(src, dst))
    lens, _ = _compact_sizes(case)
    table = s["block_table"].cpu().numpy().copy()
    for b, n in enumerate(lens):
        for j in range(_ceil(n, c["page"])):
            table[b, j] = to.get(int(table[b, j]), int(table[b, j]))
    out = ref.copy()
    out[len(live):] = 0
    pool = s["pool"].double()
    if src:
        out[dst] = ref[src]
        pool[torch.tensor(dst, device="cuda")] = s["pool"].double()[torch.tensor(src, device="cuda")]
    return table, out, pool, np.array([len(live)], np.int32)
