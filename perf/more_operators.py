"""Operators around a cache that is kept short and filled by drafts, measured: their plain forms and the library's calls.

  norm     RMS norms of the queries and keys of each head, their rotary positions, and the append of k and v
           to the sequences' 16-bit pages
  window   several query tokens per sequence (a ragged batch) attend to a sliding window of the paged cache and
           to its first tokens
  tree     a tree of drafted tokens per sequence attends to the cache; a token sees the cache and its ancestors
  accept   the K and V rows of each tree's accepted path moved to where the sequence goes on
  weights  the attention weights of a batch's query tokens, summed per cached position and KV head
  evict    the positions of least accumulated weight dropped, the rest gathered into new pages

With `own` false, `run` computes each in elementary torch operations; with `own` true it makes the library's calls.
The lengths and trees of a case follow from the case alone, its values from the seed.
"""

import math
import random

import numpy as np
import torch

own = False

FP16, BF16, FP8, INT8, INT4 = 0, 1, 2, 3, 4
KINDS = {"fp16": (FP16, torch.float16), "bf16": (BF16, torch.bfloat16)}
LOG2E = 1.0 / math.log(2.0)
EPS = 1e-6


# ---------------------------------------------------------------- cases

def _case(op, name, batch, hq, hkv, d, page, dtype, **more):
    c = dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, page=page, dtype=dtype, **more)
    return dict(c, name=name) if name else c


def _norm(name, batch, hq, hkv, d, page, dtype, rot, adjacent, cached, new_lo, new_hi):
    return _case("norm", name, batch, hq, hkv, d, page, dtype, rot=rot, adjacent=adjacent, cached=cached, nq_lo=new_lo, nq_hi=new_hi)


def _window(name, batch, hq, hkv, d, page, dtype, cache, len_lo, len_hi, nq_lo, nq_hi, window, sinks):
    return _case("window", name, batch, hq, hkv, d, page, dtype, cache=cache, len_lo=len_lo, len_hi=len_hi, nq_lo=nq_lo, nq_hi=nq_hi,
                 window=window, sinks=sinks)


def _tree(name, batch, hq, hkv, d, page, dtype, cache, len_lo, len_hi, nq_lo, nq_hi):
    return _case("tree", name, batch, hq, hkv, d, page, dtype, cache=cache, len_lo=len_lo, len_hi=len_hi, nq_lo=nq_lo, nq_hi=nq_hi)


def _accept(name, batch, hq, hkv, d, page, dtype, len_lo, len_hi, nq_lo, nq_hi, width):
    return _case("accept", name, batch, hq, hkv, d, page, dtype, len_lo=len_lo, len_hi=len_hi, nq_lo=nq_lo, nq_hi=nq_hi, width=width)


def _weights(name, batch, hq, hkv, d, page, dtype, cache, len_lo, len_hi, nq_lo, nq_hi, decay):
    return _case("weights", name, batch, hq, hkv, d, page, dtype, cache=cache, len_lo=len_lo, len_hi=len_hi, nq_lo=nq_lo, nq_hi=nq_hi, decay=decay)


def _evict(name, batch, hq, hkv, d, page, dtype, cache, len_lo, len_hi, budget, sinks, recent, to):
    return _case("evict", name, batch, hq, hkv, d, page, dtype, cache=cache, len_lo=len_lo, len_hi=len_hi, budget=budget, sinks=sinks,
                 recent=recent, to=to)


def listed():
    return [
        # one decode step of a serving batch whose model norms its queries and keys: latency counts
        _norm("norm-step", 32, 32, 8, 128, 16, "bf16", 128, False, 32768, 1, 1),
        # prompts of several sequences, odd lengths: bytes count
        _norm("norm-prompts", 6, 32, 4, 128, 64, "bf16", 128, False, 1001, 777, 2500),
        # a step that mixes single tokens and prompt chunks over three tiers, in a layer with a short window
        _window("window-mixed", 8, 32, 4, 128, 64, "bf16", "mixed", 500, 16384, 1, 256, 1024, 4),
        # a chunk of a long prompt over its own FP8 cache, window and first tokens: arithmetic counts
        _window("window-chunk", 1, 16, 2, 128, 64, "bf16", "fp8", 65536, 65536, 2048, 2048, 4096, 64),
        # the drafted tree of one small model's sequence: latency counts
        _tree("tree-one", 1, 14, 2, 64, 1024, "fp16", "16", 4096, 4096, 26, 26),
        # drafted trees of a serving batch, FP8 pages of 16 tokens, ragged contexts
        _tree("tree-batch", 32, 32, 8, 128, 16, "bf16", "fp8", 2048, 16384, 8, 64),
        # the accepted path of one tree
        _accept("accept-one", 1, 14, 2, 64, 1024, "fp16", 4096, 4096, 26, 26, 6),
        # the accepted paths of a large batch
        _accept("accept-batch", 256, 32, 8, 128, 16, "bf16", 100, 4000, 8, 64, 10),
        # the weights that one decode step of a serving batch gives to its cache: bytes count
        _weights("weights-step", 32, 32, 8, 128, 16, "bf16", "fp8", 8192, 32768, 1, 1, 1.0),
        # the last 32 tokens of some prompts look back over 16-bit pages: exponentials and arithmetic count
        _weights("weights-look", 4, 32, 8, 128, 64, "bf16", "16", 4096, 32768, 32, 32, 0.0),
        # one small model's sequence brought to its budget
        _evict("evict-one", 1, 14, 2, 64, 1024, "fp16", "16", 16384, 16384, 2048, 4, 256, "16"),
        # a serving batch's FP8 pages brought to their budgets: bytes count
        _evict("evict-batch", 16, 32, 8, 128, 16, "bf16", "fp8", 8192, 32768, 4096, 4, 512, "fp8"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "window", "tree", "accept", "weights", "evict"])
    hq, hkv, d, page = rng.choice([(14, 2, 64, 1024), (32, 8, 128, 16), (32, 4, 128, 64), (16, 2, 128, 64), (6, 6, 64, 48)])
    shape = (hq, hkv, d, page, rng.choice(["fp16", "bf16"]))
    if op == "norm":
        hi = _log(rng, 1, 2500)
        return _norm(None, _log(rng, 1, 6), *shape, rng.choice([16, 32, d]), rng.random() < 0.5, _log(rng, 1, 30000), rng.randint(1, hi), hi)
    cache = rng.choice(["16", "fp8", "int8", "mixed"])
    if op == "window":
        batch = _log(rng, 1, 24)
        hi = _log(rng, 64, min(32768, 200000 // batch))
        nq = _log(rng, 1, 300)
        return _window(None, batch, *shape, cache, rng.randint(0, hi), hi, rng.randint(1, nq), nq, _log(rng, 1, hi), rng.choice([0, 1, 4, 64, 200]))
    if op == "tree":
        batch = _log(rng, 1, 24)
        hi = _log(rng, 64, min(16384, 200000 // batch))
        nq = _log(rng, 1, 130)
        return _tree(None, batch, *shape, cache, rng.randint(0, hi), hi, rng.randint(1, nq), nq)
    if op == "accept":
        nq = _log(rng, 1, 100)
        hi = _log(rng, 1, 5000)
        return _accept(None, _log(rng, 1, 200), *shape, rng.randint(1, hi), hi, rng.randint(1, nq), nq, rng.randint(1, min(nq, 12)))
    batch = _log(rng, 1, 16)
    hi = _log(rng, 64, min(32768, 200000 // batch))
    if op == "weights":
        nq = _log(rng, 1, 70)
        return _weights(None, batch, *shape, rng.choice([cache, "int4"]), rng.randint(0, hi), hi, rng.randint(1, nq), nq, rng.choice([0.0, 0.9, 1.0]))
    budget = _log(rng, 16, hi)
    sinks = min(rng.choice([0, 1, 4, 64]), budget)
    return _evict(None, batch, *shape, cache, rng.randint(0, hi), hi, budget, sinks, rng.randint(0, budget - sinks), rng.choice(["16", "fp8"]))


def _rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _ends(r, n, lo, hi):
    """n values of a range, its ends first."""
    return [hi, lo][:n] + [r.randint(lo, hi) for _ in range(n - 2)]


def _lengths(case):
    """Cached tokens of each sequence, the new ones counted, and new tokens."""
    r, n = _rng(case), case["batch"]
    if case["op"] == "norm":
        new = _ends(r, n, case["nq_lo"], case["nq_hi"])
        return [r.randint(case["cached"] // 2, case["cached"]) + m for m in new], new
    lens = _ends(r, n, case["len_lo"], case["len_hi"])
    if case["op"] == "evict":
        return lens, [0] * n
    new = _ends(r, n, case["nq_lo"], case["nq_hi"])
    if case["op"] == "accept":
        return [a + m for a, m in zip(lens, new)], new
    return [max(a, m) for a, m in zip(lens, new)], new


def _parents(case):
    """Per sequence the tree's parents: a token's is one of those shortly before it, or -1 (the first has none)."""
    r = _rng(case)
    return [[-1] + [r.randint(max(-1, i - 9), i - 1) for i in range(1, m)] for m in _lengths(case)[1]]


def _paths(case):
    """Per sequence an accepted path: some tokens of the tree, in order."""
    r = _rng(case)
    return [sorted(r.sample(range(m), r.randint(0, min(m, case["width"])))) for m in _lengths(case)[1]]


def _ceil(a, b):
    return (a + b - 1) // b


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cuda(x):
    return torch.from_numpy(x).cuda()


def _starts(new):
    return _ints([0] + np.cumsum(new).tolist())


def _pages(case, lens, g, seed):
    """The sequences' pages: a pool per tier, their tables; pages lie anywhere in their pool."""
    kind, dtype = KINDS[case["dtype"]]
    p, hkv, d = case["page"], case["hkv"], case["d"]
    n_pages = np.array([_ceil(n, p) for n in lens])
    logical = np.arange(max(1, n_pages.max()))[None, :]
    used = logical < n_pages[:, None]
    age = n_pages[:, None] - 1 - logical          # 0: the newest page
    tier = {"16": np.full(used.shape, kind), "fp8": np.full(used.shape, FP8), "int8": np.full(used.shape, INT8), "int4": np.full(used.shape, INT4),
            "mixed": np.where(age < 4, kind, np.where(age < n_pages[:, None] // 2, FP8, INT8))}[case["cache"]]
    tier = np.where(used, tier, 0)
    table = np.zeros(used.shape, np.int64)
    perm = np.random.default_rng(int(seed))
    pools = {}
    for c in (kind, FP8, INT8, INT4):
        n = int((used & (tier == c)).sum())
        if n == 0:
            continue
        table[used & (tier == c)] = perm.permutation(n)
        shape = (n, 2, hkv, p, d)
        if c == kind:
            pools[c] = (_randn(shape, dtype, g), None)
        elif c == FP8:
            codes = torch.randn(shape, generator=g, device="cuda").mul_(100.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
            pools[c] = (codes, 0.008 + 0.004 * torch.rand((n, 2, hkv), generator=g, device="cuda"))
        elif c == INT8:
            codes = torch.randn(shape, generator=g, device="cuda").mul_(30.0).round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
            pools[c] = (codes, 0.025 + 0.015 * torch.rand((n, 2, hkv), generator=g, device="cuda"))
        else:
            codes = torch.randint(0, 256, shape[:-1] + (d // 2,), generator=g, device="cuda", dtype=torch.uint8)
            meta = torch.rand(shape[:-1] + (d // 32, 2), generator=g, device="cuda")
            pools[c] = (codes, torch.stack([0.2 + 0.1 * meta[..., 0], -1.5 - meta[..., 1]], -1).half())
    return dict(kind=kind, dtype=dtype, max_pages=used.shape[1], pools=pools, page_codec=_cuda(tier.astype(np.uint8)),
                block_table=_cuda(table.astype(np.int32)), seq_lens=_ints(lens))


def prepare(case, seed):
    return {"norm": _prepare_norm, "window": _prepare_queries, "tree": _prepare_tree, "accept": _prepare_accept, "weights": _prepare_weights,
            "evict": _prepare_evict}[case["op"]](case, seed)


def _own_pages(case, seed):
    """Tables of sequences of which only the last pages, the ones written, lie in the pool."""
    lens, new = _lengths(case)
    p = case["page"]
    max_pages = _ceil(max(lens), p)
    first = [(a - n) // p for a, n in zip(lens, new)]
    last = [_ceil(n, p) for n in lens]
    n_slots = sum(l - f for f, l in zip(first, last))
    table = np.zeros((case["batch"], max_pages), np.int32)
    perm, k = np.random.default_rng(int(seed)).permutation(n_slots), 0
    for i in range(case["batch"]):
        table[i, first[i]:last[i]] = perm[k:k + last[i] - first[i]]
        k += last[i] - first[i]
    return lens, new, max_pages, table, n_slots


def _prepare_norm(case, seed):
    g = _gen(seed)
    kind, dtype = KINDS[case["dtype"]]
    p, hq, hkv, d, half = case["page"], case["hq"], case["hkv"], case["d"], case["rot"] // 2
    lens, new, max_pages, table, n_slots = _own_pages(case, seed)
    total = sum(new)
    qkv = _randn((total, (hq + 2 * hkv) * d), dtype, g) * 3.0                         # a fused projection's rows
    at = torch.cat([torch.arange(a - n, a, device="cuda") for a, n in zip(lens, new)])
    return dict(case=case, kind=kind, dtype=dtype, max_pages=max_pages, q=qkv[:, :hq * d].view(total, hq, d),
                k=qkv[:, hq * d:(hq + hkv) * d].view(total, hkv, d), v=qkv[:, (hq + hkv) * d:].view(total, hkv, d),
                q_start=_starts(new), seq_lens=_ints(lens), positions=at.to(torch.int32)[None].contiguous(),
                inv_freq=torch.tensor([10000.0 ** (-i / half) for i in range(half)], dtype=torch.float64, device="cuda"),
                q_weight=1.0 + 0.3 * torch.randn(d, generator=g, device="cuda"), k_weight=1.0 + 0.3 * torch.randn(d, generator=g, device="cuda"),
                pool=_randn((n_slots, 2, hkv, p, d), dtype, g), page_codec=torch.full((case["batch"], max_pages), kind, dtype=torch.uint8, device="cuda"),
                block_table=_cuda(table))


def _prepare_queries(case, seed):
    g = _gen(seed)
    lens, new = _lengths(case)
    s = _pages(case, lens, g, seed)
    return dict(s, case=case, nq_max=max(new), q=_randn((sum(new), case["hq"], case["d"]), s["dtype"], g), q_start=_starts(new),
                scale=1.0 / math.sqrt(case["d"]))


def _prepare_tree(case, seed):
    s = _prepare_queries(case, seed)
    words = _ceil(s["nq_max"], 32)
    rows = []
    for parents in _parents(case):
        seen = []
        for i, a in enumerate(parents):
            seen.append((1 << i) | (seen[a] if a >= 0 else 0))
        rows += [[(x >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for x in seen]
    return dict(s, tree_mask=_cuda(np.array(rows, np.uint32).view(np.int32)))


def _prepare_accept(case, seed):
    g = _gen(seed)
    kind, dtype = KINDS[case["dtype"]]
    lens, new, max_pages, table, n_slots = _own_pages(case, seed)
    paths = _paths(case)
    path = np.full((case["batch"], case["width"]), -1, np.int32)
    for i, x in enumerate(paths):
        path[i, :len(x)] = x
    return dict(case=case, kind=kind, dtype=dtype, max_pages=max_pages, q_start=_starts(new), seq_lens=_ints(lens), path=_cuda(path),
                n_path=_ints([len(x) for x in paths]), pool=_randn((n_slots, 2, case["hkv"], case["page"], case["d"]), dtype, g),
                page_codec=torch.full((case["batch"], max_pages), kind, dtype=torch.uint8, device="cuda"), block_table=_cuda(table))


def _prepare_weights(case, seed):
    """The attention has run: its log-sums are at hand, and what was accumulated before."""
    s, c = _prepare_queries(case, seed), case
    lens, new = _lengths(case)
    grp, d, t = c["hq"] // c["hkv"], c["d"], 0
    lse2 = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    for b, (n, m) in enumerate(zip(lens, new)):
        keys = _keys_of(s, b, n, torch.float32)                                       # [Hkv, n, D]
        q = s["q"][t:t + m].float().view(m, c["hkv"], grp, d).permute(1, 2, 0, 3)
        x = torch.matmul(q.reshape(c["hkv"], grp * m, d), keys.transpose(1, 2)).mul_(s["scale"]).view(c["hkv"], grp, m, n)
        x.masked_fill_(torch.arange(n, device="cuda") > n - m + torch.arange(m, device="cuda")[:, None], -math.inf)
        lse2[t:t + m] = (torch.logsumexp(x, -1) * LOG2E).permute(2, 0, 1).reshape(m, c["hq"])
        t += m
    rows = s["max_pages"] * c["page"]
    g = _gen(seed + 1)
    return dict(s, lse2=lse2, weights=torch.rand((c["batch"], c["hkv"], rows), generator=g, device="cuda") / 64.0)


def _prepare_evict(case, seed):
    g = _gen(seed)
    c = case
    lens, _ = _lengths(case)
    s = _pages(case, lens, g, seed)
    rows, p, d = s["max_pages"] * c["page"], c["page"], c["d"]
    # few positions hold most of the weight; many were hardly looked at, and share a value
    w = torch.exp(2.0 * torch.randn((c["batch"], c["hkv"], rows), generator=g, device="cuda")) / 1024.0
    w = torch.where(w < 2e-4, 0.0, w)
    to = s["kind"] if c["to"] == "16" else FP8
    pages = _ceil(c["budget"], p)
    n_dst = c["batch"] * pages + 3
    dst_table = np.random.default_rng(int(seed) + 1).permutation(n_dst)[:c["batch"] * pages].reshape(c["batch"], pages).astype(np.int32)
    shape = (n_dst, 2, c["hkv"], p, d)
    dst = (torch.zeros(shape, dtype=s["dtype"] if to != FP8 else torch.uint8, device="cuda"),
           torch.zeros(shape[:3], device="cuda") if to == FP8 else None)
    return dict(s, case=case, weights=w, to=to, dst=dst, dst_table=_cuda(dst_table), dst_pages=pages)


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "window": _own_attention, "tree": _own_attention, "accept": _own_accept, "weights": _own_weights,
                "evict": _own_evict}[op](state)
    return {"norm": _plain_norm, "window": _plain_attention, "tree": _plain_attention, "accept": _plain_accept, "weights": _plain_weights,
            "evict": _plain_evict}[op](state)


def _argus():
    import mixed_precision_paged_argus_gb300.argus as argus
    return argus


def _geom(argus, c):
    return argus.geom(c["hq"], c["hkv"], c["d"], c["page"])


def _pools(argus, s):
    return [argus.Pool(k, codes, meta, codes.shape[0]) for k, (codes, meta) in s["pools"].items()]


def _own_norm(s):
    argus, c = _argus(), s["case"]
    q_out = torch.empty(s["q"].shape, dtype=s["dtype"], device="cuda")
    pool = argus.Pool(s["kind"], s["pool"], None, s["pool"].shape[0])
    argus.norm_rope_append(_geom(argus, c), s["q"], s["k"], s["v"], q_out, s["q_start"], s["seq_lens"], s["positions"], s["inv_freq"], pool,
                           s["page_codec"], s["block_table"], s["max_pages"], s["q_weight"], s["k_weight"], EPS, adjacent=c["adjacent"])
    return q_out, s["pool"]


def _own_attention(s):
    argus, c = _argus(), s["case"]
    out = torch.empty(s["q"].shape, dtype=s["dtype"], device="cuda")
    lse2 = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    args = argus.extend_args(_geom(argus, c), s["q"], s["q_start"], _pools(argus, s), s["page_codec"], s["block_table"], s["seq_lens"],
                             s["max_pages"], s["scale"], out, lse2_out=lse2)
    ws = torch.empty(argus.extend_workspace_bytes(args), dtype=torch.uint8, device="cuda")
    if c["op"] == "tree":
        argus.paged_tree_attn(args, ws, s["tree_mask"])
    else:
        argus.paged_window_extend_attn(args, ws, c["window"], c["sinks"])
    return out, lse2


def _own_accept(s):
    argus, c = _argus(), s["case"]
    pool = argus.Pool(s["kind"], s["pool"], None, s["pool"].shape[0])
    lens = torch.empty_like(s["seq_lens"])
    argus.accept_tokens(_geom(argus, c), pool, s["page_codec"], s["block_table"], s["max_pages"], s["q_start"], s["seq_lens"], s["path"],
                        s["n_path"], lens)
    return s["pool"], lens


def _own_weights(s):
    argus, c = _argus(), s["case"]
    args = argus.extend_args(_geom(argus, c), s["q"], s["q_start"], _pools(argus, s), s["page_codec"], s["block_table"], s["seq_lens"],
                             s["max_pages"], s["scale"], None, lse2_out=s["lse2"])
    argus.attn_weights(args, s["weights"], decay=c["decay"])
    return s["weights"]


def _own_evict(s):
    argus, c = _argus(), s["case"]
    lens = torch.empty_like(s["seq_lens"])
    kept = torch.empty((c["batch"], c["hkv"], c["budget"]), dtype=torch.int32, device="cuda")
    weights = torch.empty_like(s["weights"])
    dst = argus.Pool(s["to"], s["dst"][0], s["dst"][1], s["dst"][0].shape[0])
    argus.evict_tokens(_geom(argus, c), _pools(argus, s), s["page_codec"], s["block_table"], s["seq_lens"], s["max_pages"], s["weights"],
                       c["budget"], c["sinks"], c["recent"], dst, s["dst_table"], s["dst_pages"], lens, kept, weights)
    return _evicted(s, lens, kept, weights)


def _evicted(s, lens, kept, weights):
    codes, meta = s["dst"]
    if s["to"] == FP8:
        return lens, kept, weights, codes.view(torch.float8_e4m3fn), meta
    return lens, kept, weights, codes


# ---- norm, plainly: the angles in 64 bits (far positions), the rest in 32

def _normed(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _turned(x, cos, sin, rot, adjacent):
    if adjacent:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _token_rows(s):
    """Row and cached position of each new token."""
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    row = torch.repeat_interleave(torch.arange(n.shape[0], device="cuda"), n, output_size=s["q"].shape[0])
    return row, (s["seq_lens"].long() - n)[row] + torch.arange(s["q"].shape[0], device="cuda") - s["q_start"].long()[row]


def _plain_norm(s):
    c = s["case"]
    angle = s["positions"][0].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q_out = _turned(_normed(s["q"], s["q_weight"]), cos, sin, c["rot"], c["adjacent"]).to(s["dtype"])
    k = _turned(_normed(s["k"], s["k_weight"]), cos, sin, c["rot"], c["adjacent"]).to(s["dtype"])
    row, at = _token_rows(s)
    slot = s["block_table"][row, at // c["page"]].long()
    s["pool"][slot, 0, :, at % c["page"]] = k
    s["pool"][slot, 1, :, at % c["page"]] = s["v"]
    return q_out, s["pool"]


# ---- attention, plainly: the pages' values gathered in 32 bits, padded scores, masked softmax

def _values(codec, codes, meta):
    if codec == FP8:
        return codes.view(torch.float8_e4m3fn).float() * meta[..., None, None]
    if codec == INT8:
        return codes.view(torch.int8).float() * meta[..., None, None]
    if codec == INT4:
        x = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, 32))
        return (x * meta[..., 0].float()[..., None] + meta[..., 1].float()[..., None]).flatten(-2)
    return codes.float()


def _gathered(s):
    """K and V of every sequence in 32 bits, [2, B, Hkv, positions, D]."""
    c, mp = s["case"], s["max_pages"]
    pages = torch.zeros((c["batch"], mp, 2, c["hkv"], c["page"], c["d"]), dtype=torch.float32, device="cuda")
    used = torch.arange(mp, device="cuda")[None, :] < (s["seq_lens"][:, None] + c["page"] - 1) // c["page"]
    for codec, (codes, meta) in s["pools"].items():
        at = used & (s["page_codec"] == codec)
        slots = s["block_table"][at].long()
        pages[at] = _values(codec, codes[slots], None if meta is None else meta[slots])
    return pages.permute(2, 0, 3, 1, 4, 5).reshape(2, c["batch"], c["hkv"], mp * c["page"], c["d"])


def _padded(s):
    """Rows of the padded batch [B, nq], the new tokens' counts, and which rows are real."""
    first, n = s["q_start"][:-1].long(), (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(s["nq_max"], device="cuda")
    return (first[:, None] + i).clamp(max=s["q"].shape[0] - 1), n, i < n[:, None]


def _scores(s, keys, rows):
    c = s["case"]
    b, hkv, d, nq, grp = c["batch"], c["hkv"], c["d"], s["nq_max"], c["hq"] // c["hkv"]
    q = s["q"][rows].float().view(b, nq, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, nq * grp, d)
    return torch.matmul(q, keys.transpose(2, 3)).mul_(s["scale"]).view(b, hkv, nq, grp, -1)


def _visible(s, rows, n):
    """Which positions each row of the padded batch sees, [B, nq, positions]."""
    c, b, nq = s["case"], s["case"]["batch"], s["nq_max"]
    key = torch.arange(s["max_pages"] * c["page"], device="cuda")
    base = s["seq_lens"].long() - n
    at = base[:, None] + torch.arange(nq, device="cuda")
    if c["op"] != "tree":
        see = key <= at[..., None]
        if c["op"] == "window":
            see &= (key > at[..., None] - c["window"]) | (key < c["sinks"])
        return see
    j = (key - base[:, None])[:, None].expand(b, nq, -1)                              # the tree's tokens follow the cache
    word = torch.gather(s["tree_mask"][rows].long(), 2, (j >> 5).clamp(0, s["tree_mask"].shape[1] - 1))
    return (j < 0) | ((j < n[:, None, None]) & ((word >> (j & 31) & 1) == 1))


def _plain_attention(s):
    c = s["case"]
    b, hq, hkv, d, nq = c["batch"], c["hq"], c["hkv"], c["d"], s["nq_max"]
    kv = _gathered(s)
    rows, n, real = _padded(s)
    scores = _scores(s, kv[0], rows)
    scores.masked_fill_(~_visible(s, rows, n)[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = scores.sum(-1, keepdim=True)
    o = torch.matmul(scores.view(b, hkv, nq * (hq // hkv), -1), kv[1]).view(b, hkv, nq, hq // hkv, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse2 = ((top + total.log()) * LOG2E).squeeze(-1)
    out = o.permute(0, 2, 1, 3, 4).reshape(b, nq, hq, d)[real]
    return out.to(s["dtype"]), lse2.permute(0, 2, 1, 3).reshape(b, nq, hq)[real]


def _plain_accept(s):
    c = s["case"]
    p, width = c["page"], c["width"]
    base = (s["seq_lens"] - (s["q_start"][1:] - s["q_start"][:-1])).long()
    k = torch.arange(width, device="cuda")
    real = k < s["n_path"][:, None]
    row = torch.arange(c["batch"], device="cuda")[:, None].expand(-1, width)[real]
    src = (base[:, None] + s["path"])[real]
    dst = (base[:, None] + k)[real]
    table = s["block_table"].long()
    s["pool"][table[row, dst // p], :, :, dst % p] = s["pool"][table[row, src // p], :, :, src % p]
    return s["pool"], (base + s["n_path"]).to(torch.int32)


def _plain_weights(s):
    c = s["case"]
    keys = _gathered(s)[0]
    rows, n, real = _padded(s)
    x = _scores(s, keys, rows)                                                        # [B, Hkv, nq, G, positions]
    lse = s["lse2"][rows].view(c["batch"], s["nq_max"], c["hkv"], -1).permute(0, 2, 1, 3)
    x = x.mul_(LOG2E).sub_(lse[..., None]).exp2_()
    see = _visible(s, rows, n) & real[..., None]
    x.masked_fill_(~see[:, None, :, None, :], 0.0)
    at = torch.arange(x.shape[-1], device="cuda") < s["seq_lens"][:, None]
    s["weights"].copy_(torch.where(at[:, None], s["weights"] * c["decay"] + x.sum((2, 3)), s["weights"]))
    return s["weights"]


def _plain_evict(s):
    c = s["case"]
    b, hkv, p, d, budget = c["batch"], c["hkv"], c["page"], c["d"], c["budget"]
    old = s["seq_lens"].long()
    lens = old.clamp(max=budget)
    j = torch.arange(s["weights"].shape[-1], device="cuda")
    worth = torch.where((j < c["sinks"]) | (j >= old[:, None] - c["recent"]), math.inf, 0.0)[:, None] + s["weights"]
    worth = torch.where((j < old[:, None])[:, None], worth, -math.inf)
    best = torch.sort(worth, dim=-1, descending=True, stable=True).indices[..., :budget]
    if best.shape[-1] < budget:
        best = torch.cat([best, best.new_zeros(b, hkv, budget - best.shape[-1])], -1)
    i = torch.arange(budget, device="cuda")
    real = (i < lens[:, None])[:, None].expand(b, hkv, budget)
    far = j.shape[0]
    kept = torch.where(real, best, far).sort(-1).values
    at = torch.where(real, kept, 0)
    row = torch.arange(b, device="cuda")[:, None, None].expand_as(at)
    head = torch.arange(hkv, device="cuda")[None, :, None].expand_as(at)
    page = at // p
    tier, slot = s["page_codec"][row, page].long(), s["block_table"][row, page].long()
    x = torch.zeros((b, hkv, s["dst_pages"] * p, 2, d), device="cuda")
    for codec, (codes, meta) in s["pools"].items():
        mine = (real & (tier == codec)).nonzero(as_tuple=True)
        rows = (slot[mine], slice(None), head[mine], at[mine] % p)
        x[mine] = _values(codec, codes[rows][:, :, None], None if meta is None else meta[rows[:3]])[:, :, 0]
    x = x.view(b, hkv, s["dst_pages"], p, 2, d).permute(0, 2, 4, 1, 3, 5)              # [B, pages, 2, Hkv, P, D]
    written = torch.arange(s["dst_pages"], device="cuda") < ((lens + p - 1) // p)[:, None]
    to = s["dst_table"].long()[written]
    x = x[written]
    codes, meta = s["dst"]
    if s["to"] == FP8:
        scale = x.abs().amax((-1, -2)) / 448.0
        codes[to] = torch.where(scale[..., None, None] > 0, x / scale[..., None, None], 0.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        meta[to] = scale
    else:
        codes[to] = x.to(codes.dtype)
    weights = torch.zeros_like(s["weights"])
    m = min(budget, weights.shape[-1])
    weights[..., :m] = torch.where(real, torch.gather(s["weights"], 2, at), 0.0)[..., :m]
    return _evicted(s, lens.to(torch.int32), torch.where(real, kept, -1).to(torch.int32), weights)


# ---------------------------------------------------------------- what a pass cannot do without

def _bytes_per_value(c, n):
    """Bytes of a cached value, of a sequence's newest n positions."""
    if c["cache"] == "mixed":
        return 1.0 + min(n, 4 * c["page"]) / max(1, n)
    return {"16": 2.0, "fp8": 1.0, "int8": 1.0, "int4": 0.625}[c["cache"]]


def work(case):
    c, op = case, case["op"]
    lens, new = _lengths(c)
    total, row = sum(new), c["hkv"] * c["d"]
    if op == "norm":
        return {"bytes": total * (4.0 * (c["hq"] + 2 * c["hkv"]) * c["d"] + 4), "flops": total * (c["hq"] + c["hkv"]) * (4.0 * c["d"] + 3 * c["rot"])}
    if op == "accept":
        rows = sum(sum(1 for k, x in enumerate(path) if k != x) for path in _paths(c))
        return {"bytes": 8.0 * row * rows + 16.0 * c["batch"], "flops": 0}
    if op == "evict":
        kept = sum(min(n, c["budget"]) for n in lens)
        wide = _ceil(max(max(lens), 1), c["page"]) * c["page"]
        per = 2.0 if c["to"] == "16" else 1.0
        return {"bytes": 2 * row * kept * (per + _bytes_per_value(c, c["budget"])) + 4.0 * c["hkv"] * (sum(lens) + c["batch"] * (wide + c["budget"])), "flops": 0}
    if op == "weights":
        pairs = sum(n * m - m * (m - 1) // 2 for n, m in zip(lens, new))
        keys = sum(row * n * _bytes_per_value(c, n) for n in lens)
        return {"bytes": keys + (8.0 if c["decay"] else 4.0) * c["hkv"] * sum(lens) + total * c["hq"] * (2 * c["d"] + 4), "flops": 2.0 * c["hq"] * c["d"] * pairs}
    pairs, cached = 0, 0
    for b, (n, m) in enumerate(zip(lens, new)):
        if op == "window":
            w, k = c["window"], c["sinks"]
            seen = [min(t, w) + max(0, min(k, t - w)) for t in range(n - m + 1, n + 1)]
            pairs += sum(seen)
            near = min(n, w + m - 1)
            reach = near + min(k, n - near)
        else:
            depth = []
            for a in _parents(c)[b]:
                depth.append(1 + (depth[a] if a >= 0 else 0))
            pairs += m * (n - m) + sum(depth)
            reach = n
        cached += 2 * row * reach * _bytes_per_value(c, reach)
    return {"bytes": cached + total * c["hq"] * (4 * c["d"] + 4), "flops": 4.0 * c["hq"] * c["d"] * pairs}


# ---------------------------------------------------------------- the definitions in 64 bits

def _keys_of(s, b, n, dtype, which=0):
    """One sequence's keys (or values, which = 1), [Hkv, n, D], page by page of its table."""
    c = s["case"]
    p, n_pages = c["page"], _ceil(n, c["page"])
    tiers, slots = s["page_codec"][b, :n_pages], s["block_table"][b, :n_pages].long()
    x = torch.zeros((n_pages, c["hkv"], p, c["d"]), dtype=dtype, device="cuda")
    for k, (codes, meta) in s["pools"].items():
        at = (tiers == k).nonzero().squeeze(1)
        y = codes[slots[at], which]
        if k == INT4:
            low = torch.empty(y.shape[:-1] + (c["d"],), dtype=dtype, device="cuda")
            low[..., 0::2], low[..., 1::2] = (y % 16).to(dtype), (y // 16).to(dtype)
            m = meta[slots[at], which].to(dtype).repeat_interleave(32, -2)
            y = low * m[..., 0] + m[..., 1]
        else:
            y = y.view({FP8: torch.float8_e4m3fn, INT8: torch.int8}.get(k, y.dtype)).to(dtype)
            if meta is not None:
                y = y * meta[slots[at], which].to(dtype)[..., None, None]
        x[at] = y
    return x.transpose(0, 1).reshape(c["hkv"], n_pages * p, c["d"])[:, :n]


def exact(case, seed):
    return {"norm": _exact_norm, "window": _exact_attention, "tree": _exact_attention, "accept": _exact_accept, "weights": _exact_weights,
            "evict": _exact_evict}[case["op"]](case, seed)


def _exact_norm(case, seed):
    s, c = prepare(case, seed), case
    half, f64 = c["rot"] // 2, torch.float64
    i = torch.arange(half, device="cuda")
    one, two = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + half)
    turn = torch.polar(torch.ones((), dtype=f64, device="cuda"), s["positions"][0].to(f64)[:, None] * s["inv_freq"])

    def form(x, w):
        y = x.to(f64)
        y = y / ((y ** 2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * w.to(f64)
        z = torch.complex(y[..., one], y[..., two]) * turn[:, None]
        y[..., one], y[..., two] = z.real, z.imag
        return y

    lens, new = _lengths(case)
    pool, k, t, p = s["pool"].to(f64), form(s["k"], s["k_weight"]), 0, c["page"]
    for b, (a, n) in enumerate(zip(lens, new)):
        for page in range((a - n) // p, _ceil(a, p)):
            lo, hi = max(a - n, page * p), min(a, (page + 1) * p)
            rows, at = slice(lo - page * p, hi - page * p), slice(t + lo - (a - n), t + hi - (a - n))
            pool[int(s["block_table"][b, page]), 0, :, rows] = k[at].transpose(0, 1)
            pool[int(s["block_table"][b, page]), 1, :, rows] = s["v"][at].to(f64).transpose(0, 1)
        t += n
    return form(s["q"], s["q_weight"]), pool


def _exact_attention(case, seed):
    """Some rows of one sequence and KV head at a time, over the positions that any of them sees."""
    s, c = prepare(case, seed), case
    lens, new = _lengths(case)
    grp, f64 = c["hq"] // c["hkv"], torch.float64
    out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
    lse2 = torch.full(s["q"].shape[:2], -math.inf, dtype=f64, device="cuda")
    t0 = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        kv = [_keys_of(s, b, n, f64, which) for which in (0, 1)]
        see = torch.zeros((m, n), dtype=torch.bool, device="cuda")
        if c["op"] == "tree":
            seen = np.zeros((m, n), bool)
            seen[:, :n - m] = True
            for i, a in enumerate(_parents(case)[b]):
                seen[i, n - m:] = seen[a, n - m:] if a >= 0 else False
                seen[i, n - m + i] = True
            see = _cuda(seen)
        else:
            for i in range(m):
                at = n - m + i
                see[i, :min(c["sinks"], at + 1)] = True
                see[i, max(0, at - c["window"] + 1):at + 1] = True
        step = max(1, (1 << 27) // (n * grp))
        for r in range(0, m, step):
            k = see[r:r + step].any(0).nonzero().squeeze(1)
            hide = ~see[r:r + step][:, k][:, None]
            rows = slice(t0 + r, t0 + min(m, r + step))
            for h in range(c["hkv"]):
                q = s["q"][rows, h * grp:(h + 1) * grp].to(f64)
                x = torch.einsum("tgd,nd->tgn", q, kv[0][h][k]) * s["scale"]
                x = x.masked_fill(hide, -math.inf)
                lse = torch.logsumexp(x, -1)
                out[rows, h * grp:(h + 1) * grp] = torch.einsum("tgn,nd->tgd", torch.exp(x - lse[..., None]), kv[1][h][k])
                lse2[rows, h * grp:(h + 1) * grp] = lse / math.log(2.0)
        t0 += m
    return out, lse2


def _exact_accept(case, seed):
    s, c = prepare(case, seed), case
    lens, new = _lengths(case)
    p, table = c["page"], s["block_table"].cpu().numpy()
    pool, out, paths = s["pool"].double(), [], _paths(case)
    to, frm = [], []
    for b, (n, m) in enumerate(zip(lens, new)):
        path = paths[b]
        for k, x in enumerate(path):
            frm.append((int(table[b, (n - m + x) // p]), (n - m + x) % p))
            to.append((int(table[b, (n - m + k) // p]), (n - m + k) % p))
        out.append(n - m + len(path))
    if to:
        a, z = _cuda(np.array(frm)), _cuda(np.array(to))
        pool[z[:, 0], :, :, z[:, 1]] = s["pool"].double()[a[:, 0], :, :, a[:, 1]]
    return pool, np.array(out, np.int32)


def _exact_weights(case, seed):
    s, c = prepare(case, seed), case
    lens, new = _lengths(case)
    grp, f64, t0 = c["hq"] // c["hkv"], torch.float64, 0
    out = s["weights"].to(f64)
    for b, (n, m) in enumerate(zip(lens, new)):
        keys = _keys_of(s, b, n, f64)
        later = torch.arange(n, device="cuda") > (n - m + torch.arange(m, device="cuda"))[:, None]
        for h in range(c["hkv"]):
            rows = (slice(t0, t0 + m), slice(h * grp, (h + 1) * grp))
            x = torch.einsum("tgd,nd->tgn", s["q"][rows].to(f64), keys[h]) * (s["scale"] / math.log(2.0)) - s["lse2"][rows].to(f64)[..., None]
            x = torch.pow(2.0, x).masked_fill(later[:, None], 0.0)
            out[b, h, :n] = out[b, h, :n] * c["decay"] + x.sum((0, 1))
        t0 += m
    return out


def _exact_evict(case, seed):
    """The positions in order of worth on the host, a KV head at a time."""
    s, c = prepare(case, seed), case
    lens, _ = _lengths(case)
    p, d, budget = c["page"], c["d"], c["budget"]
    w = s["weights"].cpu().numpy()
    kept = np.full((c["batch"], c["hkv"], budget), -1, np.int32)
    weights = np.zeros(w.shape)
    pool = s["dst"][0].double() if s["to"] != FP8 else s["dst"][0].view(torch.float8_e4m3fn).double()
    meta = None if s["to"] != FP8 else s["dst"][1].double()
    table = s["dst_table"].cpu().numpy()
    for b, n in enumerate(lens):
        m, lo = min(n, budget), min(n, c["sinks"])
        pages = _ceil(m, p)
        x = torch.zeros((2, c["hkv"], pages * p, d), dtype=torch.float64, device="cuda")
        both = [_keys_of(s, b, n, torch.float64, which) for which in (0, 1)]
        for h in range(c["hkv"]):
            at = np.arange(n)
            if n > budget:
                mid = np.arange(lo, n - c["recent"])
                best = mid[np.lexsort((mid, -w[b, h, mid]))][:budget - lo - c["recent"]]
                at = np.sort(np.concatenate([np.arange(lo), best, np.arange(n - c["recent"], n)]))
            kept[b, h, :m] = at
            weights[b, h, :m] = w[b, h, at]
            for which in (0, 1):
                x[which, h, :m] = both[which][h][_cuda(at)]
        to = torch.from_numpy(table[b, :pages].astype(np.int64)).cuda()
        x = x.view(2, c["hkv"], pages, p, d).permute(2, 0, 1, 3, 4)
        if s["to"] == FP8:
            scale = x.abs().amax((-1, -2)) / 448.0
            meta[to] = scale
            x = x / torch.where(scale > 0, scale, 1.0)[..., None, None]
        pool[to] = x
    out = (np.minimum(np.array(lens), budget).astype(np.int32), kept, weights, pool)
    return out + (meta,) if s["to"] == FP8 else out
