"""Host-side checks of window and tree attention, head norms, accepted paths, attention weights and eviction: refusals
before any CUDA call, what is launched, and oracle pins."""

import ctypes
import math

import numpy as np
import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus
import oracle
from oracle import codecs as C
from test_cache_ops_cpu import INVALID, OK, UNSUPPORTED, WORKSPACE, _extend, _lib, _pools
from test_cache_refusals_cpu import _Called, _Library, extend, i32, pool_of, rope
from test_launches_cpu import run_with_fakes

# ---- refusals: every pointer below is a made-up, aligned number that no call may touch


def _window(w=100, sinks=4, ws=64, ws_bytes=1 << 40, **kw):
    a = _extend(**kw)
    return _lib().argus_paged_window_extend_attn(ctypes.byref(a), w, sinks, ws, ws_bytes, None)


def _tree(mask=64, words=1, ws=64, ws_bytes=1 << 40, **kw):
    a = _extend(**kw)
    return _lib().argus_paged_tree_attn(ctypes.byref(a), mask, words, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [_window, _tree])
@pytest.mark.parametrize("kw,status", [
    (dict(g=argus.geom(8, 3, 128, 16)), INVALID), (dict(g=argus.geom(8, 2, 96, 16)), UNSUPPORTED), (dict(g=argus.geom(18, 2, 128, 16)), UNSUPPORTED),
    (dict(causal=0), INVALID), (dict(causal=2), INVALID), (dict(batch=-1), INVALID), (dict(softmax_scale=math.nan), INVALID), (dict(q=None), INVALID),
    (dict(out=66), INVALID), (dict(seq_lens=None), INVALID), (dict(pools=[(argus.INT4_G32, 0, 64, 64, 4)]), UNSUPPORTED),
    (dict(pools=[(argus.BF16, 0, 64, None, 4)]), UNSUPPORTED), (dict(q=1 << 20), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=0), WORKSPACE)])
def test_attention_refusals(call, kw, status):
    assert call(**kw) == status
    assert _lib().argus_last_error()


def test_mask_refusals():
    for w, sinks in ((0, 4), (-1, 0), (5, -1)):
        assert _window(w, sinks) == INVALID
    assert _tree(mask=None) == INVALID and _tree(mask=66) == INVALID and _tree(words=0) == INVALID and _tree(words=-1) == INVALID
    for kw in (dict(batch=0), dict(total_q=0)):
        assert _window(**kw) == OK and _tree(**kw) == OK and _tree(mask=None, **kw) == OK
    assert _lib().argus_paged_window_extend_attn(None, 1, 0, 64, 64, None) == INVALID
    assert _lib().argus_paged_tree_attn(None, 64, 1, 64, 64, None) == INVALID


def _norm(qw=64, kw_=64, eps=1e-6, **kw):
    pool = _pools((argus.FP16, 0, 64, None, 4))
    f = dict(g=argus.geom(8, 2, 128, 16), batch=2, total_q=5, dtype=argus.FP16, rot_dim=64, adjacent=0, n_axes=3, q=64, k=64, v=64, q_out=128,
             q_stride=0, k_stride=0, v_stride=0, q_out_stride=0, positions=64, inv_freq=64, pair_axis=None, q_start=64, seq_lens=64, page_codec=64,
             block_table=64, max_pages=4, status=None)
    f.update(kw)
    a = argus.RopeArgs(pool=ctypes.cast(pool, ctypes.POINTER(argus.PoolDesc)), **f)
    return _lib().argus_norm_rope_append(ctypes.byref(a), qw, kw_, eps, None)


@pytest.mark.parametrize("kw,status", [
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID), (dict(eps=1e-31), INVALID),
    (dict(qw=66), INVALID), (dict(kw_=65), INVALID), (dict(rot_dim=40), UNSUPPORTED), (dict(q=72), INVALID), (dict(g=argus.geom(8, 2, 80, 16)), UNSUPPORTED),
    (dict(q_out=64, q_stride=2048), INVALID)])
def test_norm_refusals(kw, status):
    kw = dict(dict(q=1 << 16, k=2 << 16, v=3 << 16, q_out=4 << 16), **kw) if "q_out" not in kw else kw
    assert _norm(**kw) == status


def test_norm_without_work_is_a_no_op():
    assert _norm(batch=0) == OK and _norm(total_q=0) == OK and _lib().argus_norm_rope_append(None, 64, 64, 1e-6, None) == INVALID


def _accept(**kw):
    f = dict(g=argus.geom(8, 2, 128, 16), batch=3, pool=(argus.FP16, 0, 64, None, 4), page_codec=64, table=64, max_pages=4, q_start=64, lens=64,
             path=64, width=5, n_path=64, out=1 << 12)
    f.update(kw)
    return _lib().argus_accept_tokens(ctypes.byref(f["g"]) if f["g"] else None, f["batch"], _pools(f["pool"]) if f["pool"] else None, f["page_codec"],
                                      f["table"], f["max_pages"], f["q_start"], f["lens"], f["path"], f["width"], f["n_path"], f["out"], None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=None), INVALID), (dict(pool=None), INVALID), (dict(g=argus.geom(8, 0, 128, 16)), INVALID), (dict(g=argus.geom(8, 2, 96, 16)), UNSUPPORTED),
    (dict(g=argus.geom(8, 2, 128, 24)), UNSUPPORTED), (dict(batch=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(width=-1), INVALID),
    (dict(pool=(argus.FP8_E4M3, 0, 64, 64, 4)), UNSUPPORTED), (dict(pool=(argus.FP16, 1, 64, None, 4)), UNSUPPORTED),
    (dict(pool=(argus.FP16, 0, None, None, 4)), INVALID), (dict(pool=(argus.FP16, 0, 72, None, 4)), INVALID), (dict(pool=(argus.FP16, 0, 64, None, -1)), INVALID),
    (dict(q_start=None), INVALID), (dict(lens=None), INVALID), (dict(path=None), INVALID), (dict(n_path=None), INVALID), (dict(out=None), INVALID),
    (dict(page_codec=None), INVALID), (dict(table=None), INVALID), (dict(out=64), INVALID), (dict(lens=(1 << 12) + 8), INVALID),
    (dict(path=(1 << 12) - 56), INVALID), (dict(table=(1 << 12) - 40), INVALID), (dict(q_start=(1 << 12) - 12), INVALID)])
def test_accept_refusals(kw, status):
    assert _accept(**kw) == status
    assert _accept(batch=0, **{k: v for k, v in kw.items() if k in ("q_start", "lens")}) == OK


def _weights(weights=1 << 24, row_len=64, decay=1.0, **kw):
    a = _extend(**dict(dict(lse2_out=64, out=None), **kw))
    return _lib().argus_attn_weights(ctypes.byref(a), weights, row_len, decay, None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=argus.geom(8, 3, 128, 16)), INVALID), (dict(g=argus.geom(8, 2, 96, 16)), UNSUPPORTED), (dict(g=argus.geom(18, 2, 128, 16)), UNSUPPORTED),
    (dict(g=argus.geom(8, 2, 128, 24)), UNSUPPORTED), (dict(q_dtype=2), INVALID), (dict(causal=2), INVALID), (dict(batch=-1), INVALID),
    (dict(batch=65536), UNSUPPORTED), (dict(total_q=2 ** 30), UNSUPPORTED), (dict(max_pages=2 ** 27), UNSUPPORTED), (dict(softmax_scale=-1.0), INVALID),
    (dict(decay=math.nan), INVALID), (dict(decay=math.inf), INVALID), (dict(row_len=63), INVALID), (dict(weights=None), INVALID), (dict(weights=66), INVALID),
    (dict(lse2_out=None), INVALID), (dict(lse2_out=66), INVALID), (dict(q=None), INVALID), (dict(q=72), INVALID), (dict(q_start=None), INVALID),
    (dict(seq_lens=None), INVALID), (dict(page_codec=None), INVALID), (dict(block_table=None), INVALID), (dict(q_stride=8), INVALID),
    (dict(q_stride=8 * 128 + 4), INVALID), (dict(pools=[(7, 0, 64, 64, 4)]), INVALID), (dict(pools=[(argus.BF16, 0, 64, None, 4)]), UNSUPPORTED),
    (dict(pools=[(argus.INT4_G32, 1, 64, 64, 4)]), UNSUPPORTED), (dict(pools=[(argus.INT2_G32, 0, 64, None, 4)]), INVALID),
    (dict(pools=[(argus.INT8, 0, 64, 64, 4)] * 2), INVALID), (dict(pools=[(argus.INT8, 0, 72, 64, 4)]), INVALID), (dict(pools=[(argus.INT8, 0, 64, 66, 4)]), INVALID),
    (dict(lse2_out=(1 << 24) + 1020), INVALID), (dict(q=(1 << 24) - 5 * 2048 + 16), INVALID), (dict(block_table=(1 << 24) - 28), INVALID)])
def test_weights_refusals(kw, status):
    assert _weights(**kw) == status


def test_weights_without_work_is_a_no_op():
    assert _weights(batch=0) == OK and _weights(max_pages=0) == OK and _lib().argus_attn_weights(None, 64, 64, 1.0, None) == INVALID


def _evict(**kw):
    f = dict(g=argus.geom(8, 2, 128, 16), batch=3, pools=[(argus.FP16, 0, 64, None, 4), (argus.FP8_E4M3, 0, 64, 64, 4)], page_codec=64, table=64, lens=64,
             max_pages=4, weights=64, row_len=64, budget=40, sinks=4, recent=8, dst=(argus.FP8_E4M3, 0, 64, 64, 9), dst_table=64, dst_pages=3, out=1 << 20,
             kept=2 << 20, w_out=3 << 20, row_out=40)
    f.update(kw)
    return _lib().argus_evict_tokens(ctypes.byref(f["g"]) if f["g"] else None, f["batch"], _pools(*f["pools"]), len(f["pools"]), f["page_codec"], f["table"],
                                     f["lens"], f["max_pages"], f["weights"], f["row_len"], f["budget"], f["sinks"], f["recent"],
                                     _pools(f["dst"]) if f["dst"] else None, f["dst_table"], f["dst_pages"], f["out"], f["kept"], f["w_out"], f["row_out"], None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=None), INVALID), (dict(dst=None), INVALID), (dict(g=argus.geom(8, 0, 128, 16)), INVALID), (dict(g=argus.geom(8, 2, 96, 16)), UNSUPPORTED),
    (dict(g=argus.geom(8, 2, 128, 24)), UNSUPPORTED), (dict(batch=-1), INVALID), (dict(batch=65536), UNSUPPORTED), (dict(max_pages=-1), INVALID),
    (dict(max_pages=2 ** 27, row_len=2 ** 31), UNSUPPORTED), (dict(budget=-1), INVALID), (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID),
    (dict(sinks=40, recent=1), INVALID), (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), INVALID), (dict(dst_pages=2), INVALID), (dict(dst_pages=-1), INVALID),
    (dict(row_len=63), INVALID), (dict(row_out=39), INVALID), (dict(dst=(argus.INT4_G32, 0, 64, 64, 9)), UNSUPPORTED), (dict(dst=(9, 0, 64, 64, 9)), INVALID),
    (dict(dst=(argus.BF16, 0, 64, None, 9)), UNSUPPORTED), (dict(dst=(argus.FP16, 1, 64, None, 9)), UNSUPPORTED), (dict(dst=(argus.FP8_E4M3, 0, 64, None, 9)), INVALID),
    (dict(dst=(argus.FP8_E4M3, 0, 72, 64, 9)), INVALID), (dict(dst=(argus.FP8_E4M3, 0, 64, 64, -1)), INVALID), (dict(pools=[(9, 0, 64, 64, 4)]), INVALID),
    (dict(pools=[(argus.INT8, 0, 64, 64, 4)] * 2), INVALID), (dict(pools=[(argus.INT8, 1, 64, 64, 4)]), UNSUPPORTED),
    (dict(pools=[(argus.INT2_G32, 0, 64, None, 4)]), INVALID), (dict(lens=None), INVALID), (dict(out=None), INVALID), (dict(weights=None), INVALID),
    (dict(page_codec=None), INVALID), (dict(table=None), INVALID), (dict(kept=None), INVALID), (dict(dst_table=None), INVALID), (dict(w_out=None), INVALID),
    (dict(out=64), INVALID), (dict(kept=64), INVALID), (dict(w_out=64 + 1532), INVALID), (dict(kept=(3 << 20) + 8), INVALID), (dict(out=(2 << 20) + 956), INVALID),
    (dict(dst_table=(1 << 20) + 8), INVALID), (dict(g=argus.geom(65535, 65535, 128, 16), batch=1, budget=10 ** 6, dst_pages=10 ** 5, row_out=10 ** 6), UNSUPPORTED)])
def test_evict_refusals(kw, status):
    assert _evict(**kw) == status


def test_evict_refuses_budgets_whose_pages_pass_32_bits():
    big = dict(batch=1, row_out=2 ** 31, sinks=0, recent=0, out=1 << 10, w_out=3 << 50, kept=1 << 50, dst_table=4 << 50)
    assert _evict(budget=2 ** 31 - 1, dst_pages=2 ** 27, **big) == UNSUPPORTED
    assert _evict(budget=2 ** 31 - 65519, dst_pages=2 ** 27 - 4094, **big) == UNSUPPORTED
    assert _evict(g=argus.geom(8, 2, 128, 2 ** 30 + 2 ** 29), max_pages=1, row_len=2 ** 31, weights=5 << 50, budget=2 ** 31 - 70000, dst_pages=2, **big) == UNSUPPORTED


def test_evict_without_work_is_a_no_op():
    assert _evict(batch=0) == OK


# ---- the binding

@pytest.fixture
def no_library(monkeypatch):
    monkeypatch.setattr(argus, "lib", lambda: _Library())
    monkeypatch.setattr(argus, "_stream_of", lambda device, stream: None)


WS = torch.zeros(64, dtype=torch.uint8)


def accept(**kw):
    f = dict(g=argus.geom(4, 2, 64, 16), pool=pool_of(argus.FP16), page_codec=torch.zeros(2, 4, dtype=torch.uint8), block_table=i32(2, 4), max_pages=4,
             q_start=i32(3), seq_lens=i32(2), path=i32(2, 5), n_path=i32(2), seq_lens_out=i32(2))
    f.update(kw)
    argus.accept_tokens(**f)


def evict(**kw):
    f = dict(g=argus.geom(4, 2, 64, 16), pools=[pool_of(argus.FP8_E4M3)], page_codec=torch.zeros(2, 4, dtype=torch.uint8), block_table=i32(2, 4),
             seq_lens=i32(2), max_pages=4, weights=torch.zeros(2, 2, 64), budget=20, sink_tokens=1, recent_tokens=2, dst=pool_of(argus.FP8_E4M3),
             dst_table=i32(2, 2), dst_pages=2, seq_lens_out=i32(2), kept=i32(2, 2, 20), weights_out=torch.zeros(2, 2, 20))
    f.update(kw)
    argus.evict_tokens(**f)


def weigh(weights=None, **kw):
    argus.attn_weights(extend(out=None, **kw), torch.zeros(2, 2, 64) if weights is None else weights)


def norm(q_weight=None, k_weight=None, eps=1e-6, **kw):
    f = dict(g=argus.geom(4, 2, 64, 16), q=torch.zeros(3, 4, 64, dtype=torch.float16), k=torch.zeros(3, 2, 64, dtype=torch.float16),
             v=torch.zeros(3, 2, 64, dtype=torch.float16), q_out=torch.zeros(3, 4, 64, dtype=torch.float16), q_start=i32(3), seq_lens=i32(2),
             positions=i32(1, 3), inv_freq=torch.zeros(32, dtype=torch.float64), pool=pool_of(argus.FP16),
             page_codec=torch.zeros(2, 4, dtype=torch.uint8), block_table=i32(2, 4), max_pages=4)
    f.update(kw)
    argus.norm_rope_append(q_weight=q_weight, k_weight=k_weight, eps=eps, **f)


def test_the_binding_takes_what_is_right(no_library):
    for call in (accept, evict, weigh, norm, rope, lambda: norm(torch.zeros(64), torch.zeros(64)), lambda: argus.paged_tree_attn(extend(), WS, i32(3, 1)),
                 lambda: argus.paged_window_extend_attn(extend(), WS, 5, 2)):
        with pytest.raises(_Called):
            call()


@pytest.mark.parametrize("call,bad", [
    (accept, [dict(path=i32(2)), dict(path=i32(3, 5)), dict(path=torch.zeros(2, 5)), dict(path=i32(2, 10)[:, ::2]), dict(n_path=i32(1)), dict(q_start=i32(2)),
              dict(seq_lens_out=i32(1)), dict(block_table=i32(2, 3)), dict(pool=argus.Pool(argus.FP16, pool_of(argus.FP16).codes, None, 5, argus.PLACE_DEVICE)),
              dict(max_pages=2 ** 32 + 4)]),
    (evict, [dict(weights=torch.zeros(2, 2, 64).double()), dict(weights=torch.zeros(2, 64)), dict(weights=torch.zeros(1, 2, 64).expand(2, 2, 64)),
             dict(weights_out=torch.zeros(2, 1, 20)), dict(weights_out=torch.zeros(2, 2, 40)[..., ::2]), dict(kept=i32(2, 2, 19)), dict(kept=torch.zeros(2, 2, 20)),
             dict(dst_table=i32(2, 1)), dict(seq_lens_out=i32(1)), dict(budget=2 ** 32 + 20), dict(sink_tokens=2 ** 32), dict(recent_tokens=-2 ** 31 - 1),
             dict(dst_pages=2 ** 32 + 2), dict(max_pages=2 ** 32 + 4), dict(page_codec=torch.zeros(2, 4)),
             dict(dst=argus.Pool(argus.FP8_E4M3, pool_of(argus.FP8_E4M3).codes, torch.zeros(3, 2, 2), 4, argus.PLACE_DEVICE))]),
    (weigh, [dict(weights=torch.zeros(2, 64)), dict(weights=torch.zeros(2, 1, 64)), dict(weights=torch.zeros(2, 2, 64).half()),
             dict(weights=torch.zeros(2, 2, 128)[..., ::2])]),
    (norm, [dict(q_weight=torch.zeros(63)), dict(k_weight=torch.zeros(64).half()), dict(q_weight=torch.zeros(128)[::2]),
            dict(q=torch.zeros(1, 4, 64, dtype=torch.float16).expand(3, 4, 64))])])
def test_the_binding_refuses_what_is_not(no_library, call, bad):
    for kw in bad:
        with pytest.raises(ValueError):
            call(**kw)


def test_the_binding_refuses_masks_of_other_shapes(no_library):
    for mask in (i32(3), i32(4, 1), torch.zeros(3, 1), i32(3, 4)[:, ::2], torch.zeros(3, 1, dtype=torch.int64)):
        with pytest.raises(ValueError):
            argus.paged_tree_attn(extend(), WS, mask)
    for w, sinks in ((2 ** 32 + 1, 0), (5, 2 ** 32)):
        with pytest.raises(ValueError, match="32 bits"):
            argus.paged_window_extend_attn(extend(), WS, w, sinks)


# ---- launches (test_launches_cpu.py has the stand-ins)

LAUNCHES = r"""
static argus_extend_args ext(argus_pool* pool) {
  argus_extend_args a;
  memset(&a, 0, sizeof a);
  a.g = (argus_geom){8, 2, 128, 16};
  a.batch = 2; a.total_q = 5; a.q_dtype = ARGUS_BF16; a.causal = 1;
  a.q = (void*)64; a.q_start = (void*)64; a.pools = pool; a.n_pools = 1; a.max_pages = 100;
  a.page_codec = (void*)64; a.block_table = (void*)64; a.seq_lens = (void*)64; a.out = (void*)(1 << 20); a.lse2_out = (void*)(2 << 20);
  a.softmax_scale = 0.5f;
  return a;
}
static argus_pool pool = {ARGUS_FP8_E4M3, 0, (void*)64, (void*)64, 400};
static int window(void) { argus_extend_args a = ext(&pool); return argus_paged_window_extend_attn(&a, 50, 4, (void*)64, (size_t)1 << 40, 0); }
static int tree(void) { argus_extend_args a = ext(&pool); return argus_paged_tree_attn(&a, (void*)64, 1, (void*)64, (size_t)1 << 40, 0); }
static int evict(void) {
  argus_geom g = {8, 2, 128, 16};
  return argus_evict_tokens(&g, 2, &pool, 1, (void*)64, (void*)64, (void*)64, 100, (void*)64, 1600, 100, 4, 8, &pool, (void*)64, 7, (void*)(1 << 20),
                            (void*)(2 << 20), (void*)(3 << 20), 100, 0, 0);
}
static int norm(void) { const argus_rope_args a = rope_args(); return argus_norm_rope_append(&a, 0, 0, 1e-6f, 0); }
static int weigh(void) { argus_extend_args a = ext(&pool); return argus_attn_weights(&a, (void*)(4 << 20), 1600, 1.f, 0); }
static int step(void) { argus_extend_args a = ext(&pool); a.total_q = 2; return argus_attn_weights(&a, (void*)(4 << 20), 1600, 1.f, 0); }
static int accept_(void) {
  argus_geom g = {8, 2, 128, 16};
  argus_pool p = {ARGUS_FP16, 0, (void*)64, 0, 400};
  return argus_accept_tokens(&g, 2, &p, (void*)64, (void*)64, 100, (void*)64, (void*)64, (void*)64, 4, (void*)64, (void*)(1 << 20), 0, 0);
}
int main(void) {
  int (*calls[])(void) = {window, tree, evict, weigh, norm, accept_, step};
  for (int c = 0; c < 7; ++c)
    for (int at = -1; at < 2; ++at) {
      fail_at = at; launches = 0; last = 0;
      const int st = calls[c]();
      printf("%d %d %d\n", st, launches, last != 0);
    }
  (void)extend; (void)rope; (void)compact;
  return 0;
}
"""


def test_a_refused_launch_ends_the_call_and_leaves_no_error(tmp_path):
    """The join reads what the attention describes, the gathering what the selection keeps: without the first kernel the
    second must not be launched; of the weights' two kernels each has sequences of its own, but one refused ends the call."""
    got = run_with_fakes(LAUNCHES, tmp_path)
    two = [(0, 2, 0), (4, 1, 0), (4, 2, 0)]
    one = [(0, 1, 0), (4, 1, 0), (0, 1, 0)]
    assert got == two * 4 + one * 3


# ---- oracle pins

def test_head_norm_oracle_is_torchs():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((5, 3, 64)), rng.standard_normal(64)
    assert np.allclose(oracle.head_norm(x, w, 1e-3), torch.nn.functional.rms_norm(torch.from_numpy(x), (64,), torch.from_numpy(w), 1e-3).numpy(), rtol=1e-13)


def _cache(rng, B, pages, Hkv, P, D):
    x = rng.standard_normal((B * pages, 2, Hkv, P, D)).astype(np.float16)
    return {C.CODEC_FP16: (x.view(np.uint16), None)}, np.arange(B * pages, dtype=np.int32).reshape(B, pages), np.zeros((B, pages), np.uint8)


def test_rules_of_sight_reduce_to_the_causal_one():
    rng = np.random.default_rng(2)
    pools, table, codec = _cache(rng, 2, 3, 1, 16, 64)
    lens, q_start = [41, 6], [0, 5, 9]
    q = rng.standard_normal((9, 2, 64))
    plain = oracle.paged_extend(q, q_start, 1, 16, pools, codec, table, lens, 0.2)
    chains = [[(1 << (i + 1)) - 1 for i in range(n)] for n in (5, 4)]
    for sees in (oracle.window_sees(1000, 0), oracle.window_sees(1, 1000), oracle.tree_sees(chains)):
        got = oracle.paged_extend(q, q_start, 1, 16, pools, codec, table, lens, 0.2, sees=sees)
        assert np.allclose(got[0], plain[0], rtol=1e-13) and np.allclose(got[1], plain[1], rtol=1e-13)
    # a window of one position is that position's value
    one = oracle.paged_extend(q, q_start, 1, 16, pools, codec, table, lens, 0.2, sees=oracle.window_sees(1, 0))[0]
    assert np.allclose(one[4, 0], pools[0][0].view(np.float16)[2, 1, 0, 40 % 16])
    # two leaves of one root do not see each other: each is a chain of its own
    masks = [[0b00001, 0b00011, 0b00101, 0b01011, 0b10101], chains[1]]
    got = oracle.paged_extend(q, q_start, 1, 16, pools, codec, table, lens, 0.2, sees=oracle.tree_sees(masks))[0]
    dense = pools[0][0].view(np.float16)[:3].astype(np.float64).transpose(1, 0, 3, 2, 4).reshape(2, 48, 64)
    keep = [*range(36), 36, 38, 40]
    s = 0.2 * dense[0, keep] @ q[4, 1]
    w = np.exp(s - s.max())
    assert np.allclose(got[4, 1], w @ dense[1, keep] / w.sum(), rtol=1e-12)


def test_weights_oracle_sums_to_the_rows():
    rng = np.random.default_rng(3)
    pools, table, codec = _cache(rng, 2, 3, 2, 16, 64)
    lens, q_start = [41, 6], [0, 5, 9]
    q = rng.standard_normal((9, 4, 64))
    for causal in (True, False):
        lse = oracle.paged_extend(q, q_start, 2, 16, pools, codec, table, lens, 0.2, causal)[1]
        w, bad, _ = oracle.attn_weights(q, q_start, lse, 2, 16, pools, codec, table, lens, 0.2, np.full((2, 2, 48), 8.0), 0.0, causal)
        assert bad == 0 and np.allclose(w[0, :, :41].sum(-1), 10) and np.allclose(w[1, :, :6].sum(-1), 8) and np.all(w[0, :, 41:] == 8)
        more, _, _ = oracle.attn_weights(q, q_start, lse, 2, 16, pools, codec, table, lens, 0.2, w, 0.5, causal)
        assert np.allclose(more[0, :, :41], 1.5 * w[0, :, :41])


def test_evict_oracle_keeps_the_heaviest():
    rng = np.random.default_rng(4)
    w = np.round(rng.random(200) * 8).astype(np.float32)
    for budget, sinks, recent in ((50, 4, 10), (200, 0, 0), (10, 10, 0), (30, 0, 30)):
        ks = oracle.evict_keep(w, 200, budget, sinks, recent)
        assert len(ks) == budget == len(set(ks)) and ks == sorted(ks)
        assert set(range(sinks)) <= set(ks) and set(range(200 - recent, 200)) <= set(ks)
        mid = [j for j in ks if sinks <= j < 200 - recent]
        out = [j for j in range(sinks, 200 - recent) if j not in ks]
        if mid and out:
            worst = min(w[j] for j in mid)
            assert worst >= max(w[j] for j in out)
            # among equals the lower positions
            assert max([j for j in mid if w[j] == worst]) < min([j for j in out if w[j] == worst], default=1000)
    assert oracle.evict_keep(np.array([np.nan, -np.inf, -0.0, 0.0, 1.0], np.float32), 5, 3, 0, 0) == [2, 3, 4]
    assert oracle.evict_keep(np.array([np.nan, -np.inf, np.nan], np.float32), 3, 2, 0, 0) == [0, 1]


def test_evict_oracle_moves_rows_as_they_are():
    rng = np.random.default_rng(5)
    pools, table, codec = _cache(rng, 1, 4, 2, 16, 64)
    w = rng.random((1, 2, 64)).astype(np.float32)
    codes, meta = C.alloc_pool(0, 2, 2, 16, 64)
    lens, kept, w_out, bad = oracle.evict_tokens(2, 16, 64, pools, codec, table, [60], w, 20, 2, 3, 0, codes, meta, np.array([[1, 0]]), 25)
    assert bad == 0 and lens[0] == 20
    flat = pools[0][0].transpose(1, 2, 0, 3, 4).reshape(2, 2, 64, 64)
    new = codes[[1, 0]].transpose(1, 2, 0, 3, 4).reshape(2, 2, 32, 64)
    for h in range(2):
        assert np.array_equal(new[:, h, :20], flat[:, h, kept[0, h]]) and np.all(new[:, h, 20:] == 0)
        assert np.array_equal(w_out[0, h], np.concatenate([w[0, h, kept[0, h]], np.zeros(5, np.float32)]))


def test_accept_oracle_keeps_the_path():
    table, codec = np.array([[5, 2, 7]], np.int32), np.zeros((1, 3), np.uint8)
    moves, lens, bad = oracle.accept_tokens([0, 10], [34], np.array([[0, 2, 3, 9]]), [4], 16, codec, table, 0, 8)
    rows = list(range(34))
    at = {(int(table[0, c // 16]), c % 16): c for c in range(48)}
    for a, z in moves:
        rows[at[z]] = rows[at[a]]
    assert bad == 0 and lens[0] == 28 and rows[24:28] == [24, 26, 27, 33] and rows[:24] == list(range(24))
