"""Host-side checks of the cache operators (ragged attention, rotary append, fork, compact):
struct layouts, refusals before any CUDA call, and oracle pins."""

import ctypes
import math
import os

import numpy as np
import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus
import oracle
from oracle import codecs as C
from test_abi_cpu import _c_layout

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


def _lib():
    if not os.path.exists(argus.lib_path()):
        from mixed_precision_paged_argus_gb300 import build
        build.build()
    return argus.lib()


@pytest.mark.parametrize("cls,struct", [(argus.ExtendArgs, "argus_extend_args"), (argus.RopeArgs, "argus_rope_args")])
def test_binding_structs_match_the_header_layout(cls, struct, tmp_path):
    names = [f[0] for f in cls._fields_]
    size, offs = _c_layout(struct, names, tmp_path)
    assert ctypes.sizeof(cls) == size
    assert [getattr(cls, n).offset for n in names] == offs


@pytest.mark.parametrize("cls,packed", [(argus.ExtendArgs, argus._EXTEND_ARGS), (argus.RopeArgs, argus._ROPE_ARGS),
                                        (argus.PoolDesc, argus._POOL_DESC)])
def test_packed_fields_land_where_the_struct_has_them(cls, packed):
    n = len(packed.unpack(bytes(packed.size)))
    a, at = cls.from_buffer_copy(packed.pack(*range(1, n + 1))), 1
    for name, kind in cls._fields_:
        x = getattr(a, name)
        if kind is argus.Geom:
            assert [getattr(x, f) for f, _ in kind._fields_] == list(range(at, at + 4))
            at += 4
            continue
        if kind is ctypes.POINTER(argus.PoolDesc):
            x = ctypes.cast(x, ctypes.c_void_p).value
        assert x == at, name
        at += 1
    assert at == n + 1 and ctypes.sizeof(a) == packed.size


# ---- refusals: every pointer below is a made-up, aligned number that no call may touch

def _pools(*descs):
    return (argus.PoolDesc * max(1, len(descs)))(*[argus.PoolDesc(*d) for d in descs])


def _extend(**kw):
    f = dict(g=argus.geom(8, 2, 128, 16), batch=2, total_q=5, q_dtype=argus.FP16, causal=1, q=64, q_stride=0, q_start=64,
             pools=[(argus.FP16, 0, 64, None, 4), (argus.FP8_E4M3, 0, 64, 64, 4)], max_pages=4, page_codec=64, block_table=64,
             seq_lens=64, out=1 << 20, lse2_out=None, status=None, softmax_scale=0.5)
    f.update(kw)
    arr = _pools(*f.pop("pools"))
    n = len(kw["pools"]) if "pools" in kw else 2
    a = argus.ExtendArgs(pools=arr, n_pools=n, **f)
    a._keep = arr
    return a


def _extend_status(ws=64, ws_bytes=1 << 40, **kw):
    a = _extend(**kw)
    return _lib().argus_paged_extend_attn(ctypes.byref(a), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=argus.geom(8, 3, 128, 16)), INVALID), (dict(g=argus.geom(0, 2, 128, 16)), INVALID),
    (dict(g=argus.geom(8, 2, 96, 16)), UNSUPPORTED), (dict(g=argus.geom(18, 2, 128, 16)), UNSUPPORTED),
    (dict(g=argus.geom(8, 2, 128, 24)), UNSUPPORTED), (dict(g=argus.geom(8, 2, 128, 0)), INVALID),
    (dict(q_dtype=2), INVALID), (dict(causal=2), INVALID), (dict(batch=-1), INVALID), (dict(total_q=-1), INVALID),
    (dict(max_pages=-1), INVALID), (dict(batch=65536), UNSUPPORTED), (dict(total_q=2 ** 30), UNSUPPORTED),
    (dict(max_pages=2 ** 27), UNSUPPORTED), (dict(softmax_scale=-1.0), INVALID), (dict(softmax_scale=math.inf), INVALID),
    (dict(softmax_scale=math.nan), INVALID), (dict(q=None), INVALID), (dict(q=72), INVALID), (dict(out=None), INVALID),
    (dict(out=66), INVALID), (dict(q_start=None), INVALID), (dict(seq_lens=None), INVALID), (dict(page_codec=None), INVALID),
    (dict(block_table=None), INVALID), (dict(q_stride=8 * 128 - 8), INVALID), (dict(q_stride=8 * 128 + 4), INVALID),
    (dict(pools=[(7, 0, 64, 64, 4)]), INVALID), (dict(pools=[(argus.INT4_G32, 0, 64, 64, 4)]), UNSUPPORTED),
    (dict(pools=[(argus.BF16, 0, 64, None, 4)]), UNSUPPORTED), (dict(pools=[(argus.FP8_E4M3, 1, 64, 64, 4)]), UNSUPPORTED),
    (dict(pools=[(argus.FP8_E4M3, 0, 64, None, 4)]), INVALID), (dict(pools=[(argus.FP8_E4M3, 0, None, 64, 4)]), INVALID),
    (dict(pools=[(argus.FP8_E4M3, 0, 72, 64, 4)]), INVALID), (dict(pools=[(argus.INT8, 0, 64, 66, 4)]), INVALID),
    (dict(pools=[(argus.INT8, 0, 64, 64, -1)]), INVALID),
    (dict(pools=[(argus.INT8, 0, 64, 64, 4), (argus.INT8, 0, 64, 64, 4)]), INVALID),
    # five tokens of 2048 bytes: out on, before and behind q, and between its strided tokens
    (dict(q=1 << 20), INVALID), (dict(q=(1 << 20) + 5 * 2048 - 16), INVALID), (dict(q=(1 << 20) - 5 * 2048 + 16), INVALID),
    (dict(q=(1 << 20) - 4096, q_stride=8192), INVALID),
    (dict(ws=None), INVALID), (dict(ws=72), INVALID), (dict(ws_bytes=0), WORKSPACE)])
def test_extend_refusals(kw, status):
    assert _extend_status(**kw) == status
    assert _lib().argus_last_error()


def test_extend_without_work_is_a_no_op():
    assert _extend_status(batch=0) == OK and _extend_status(total_q=0) == OK
    n = ctypes.c_size_t(0)
    assert _lib().argus_extend_workspace_bytes(None, ctypes.byref(n)) == INVALID
    assert _lib().argus_extend_workspace_bytes(ctypes.byref(_extend()), None) == INVALID


def _rope_status(**kw):
    pool = _pools(kw.pop("pool", (argus.FP16, 0, 64, None, 4)))
    f = dict(g=argus.geom(8, 2, 128, 16), batch=2, total_q=5, dtype=argus.FP16, rot_dim=64, adjacent=0, n_axes=3, q=64, k=64, v=64,
             q_out=128, q_stride=0, k_stride=0, v_stride=0, q_out_stride=0, positions=64, inv_freq=64, pair_axis=None, q_start=64,
             seq_lens=64, page_codec=64, block_table=64, max_pages=4, status=None)
    f.update(kw)
    a = argus.RopeArgs(pool=ctypes.cast(pool, ctypes.POINTER(argus.PoolDesc)), **f)
    return _lib().argus_rope_append(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=argus.geom(8, 3, 128, 16)), INVALID), (dict(g=argus.geom(8, 2, 80, 16)), UNSUPPORTED),
    (dict(g=argus.geom(8, 2, 128, 20)), UNSUPPORTED), (dict(dtype=argus.INT8), INVALID), (dict(batch=-1), INVALID),
    (dict(total_q=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(n_axes=0), INVALID), (dict(n_axes=5), INVALID),
    (dict(adjacent=2), INVALID), (dict(rot_dim=0), INVALID), (dict(rot_dim=144), INVALID), (dict(rot_dim=40), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q_out=None), INVALID),
    (dict(positions=None), INVALID), (dict(inv_freq=None), INVALID), (dict(q_start=None), INVALID), (dict(seq_lens=None), INVALID),
    (dict(page_codec=None), INVALID), (dict(block_table=None), INVALID), (dict(q=72), INVALID), (dict(k=72), INVALID),
    (dict(v=72), INVALID), (dict(q_out=72), INVALID), (dict(q_stride=8), INVALID), (dict(k_stride=8), INVALID),
    (dict(v_stride=260), INVALID), (dict(q_out=64, q_stride=2048), INVALID), (dict(pool=(argus.BF16, 0, 64, None, 4)), UNSUPPORTED),
    (dict(pool=(argus.FP8_E4M3, 0, 64, 64, 4)), UNSUPPORTED), (dict(pool=(argus.FP16, 1, 64, None, 4)), UNSUPPORTED),
    (dict(pool=(argus.FP16, 0, None, None, 4)), INVALID), (dict(pool=(argus.FP16, 0, 72, None, 4)), INVALID),
    (dict(pool=(argus.FP16, 0, 64, None, -1)), INVALID)])
def test_rope_refusals(kw, status):
    assert _rope_status(**kw) == status


class _Elsewhere(torch.Tensor):
    """A tensor that says it lies on the second GPU."""

    def get_device(self):
        return 1


def _call_extend(**kw):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pool = argus.Pool(argus.FP8_E4M3, torch.zeros(4, 2, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 2), 4, argus.PLACE_DEVICE)
    f = dict(g=argus.geom(8, 2, 64, 16), q=torch.zeros(3, 8, 64, dtype=torch.float16), q_start=i32(3), pools=[pool],
             page_codec=torch.zeros(2, 4, dtype=torch.uint8), block_table=i32(2, 4), seq_lens=i32(2), max_pages=4, softmax_scale=1.0,
             out=torch.zeros(3, 8, 64, dtype=torch.float16), lse2_out=torch.zeros(3, 8), status=i32(1))
    f.update({k: f[k].as_subclass(_Elsewhere) for k in kw if k in f and k != "pools"})
    if "pools" in kw:
        pool.meta = pool.meta.as_subclass(_Elsewhere)
    return argus.extend_args(**f)


@pytest.mark.parametrize("name", ["q_start", "page_codec", "block_table", "seq_lens", "out", "lse2_out", "status", "pools", "q"])
def test_binding_refuses_tensors_of_other_devices(name):
    _call_extend()
    with pytest.raises(ValueError, match="another device"):
        _call_extend(**{name: True})


def test_binding_refuses_a_device_that_is_not_current(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="not the current device"):
        argus._stream_of(1, None)
    assert argus._stream_of(0, 77) == 77
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    with pytest.raises(ValueError, match="on the GPU"):
        argus._stream_of(-1, None)


def test_rope_without_work_is_a_no_op():
    assert _rope_status(batch=0) == OK and _rope_status(total_q=0) == OK


def _fork_status(pools=((argus.FP16, 0, 64, None, 40), (argus.INT8, 0, 64, 64, 40)), ws=64, ws_bytes=1 << 40, refs=None, **kw):
    f = dict(g=argus.geom(2, 2, 64, 16), batch=3, parents=64, n_new=None, codec=argus.FP16, page_codec=64, table=64, lens=64,
             page_codec_out=128, table_out=128, lens_out=128, max_pages=4)
    f.update(kw)
    rin, rout = refs or ([64] * len(pools), [128] * len(pools))
    vp = ctypes.c_void_p
    return _lib().argus_fork_pages(ctypes.byref(f["g"]) if f["g"] else None, f["batch"], f["parents"], f["n_new"], f["codec"],
                                   _pools(*pools), len(pools), (vp * 8)(*rin), (vp * 8)(*rout), f["page_codec"], f["table"], f["lens"],
                                   f["page_codec_out"], f["table_out"], f["lens_out"], f["max_pages"], ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=None), INVALID), (dict(g=argus.geom(2, 2, 32, 16)), UNSUPPORTED), (dict(g=argus.geom(2, 2, 64, 8)), UNSUPPORTED),
    (dict(batch=-1), INVALID), (dict(batch=65536), UNSUPPORTED), (dict(max_pages=0), INVALID), (dict(codec=argus.BF16), INVALID),
    (dict(pools=()), INVALID), (dict(pools=((argus.FP16, 0, 64, None, 4),) * 2), INVALID), (dict(parents=None), INVALID),
    (dict(table=None), INVALID), (dict(table_out=64), INVALID), (dict(page_codec_out=64), INVALID), (dict(lens_out=64), INVALID),
    (dict(lens_out=None), INVALID), (dict(refs=([64, 64], [128, 64])), INVALID), (dict(refs=([64, None], [128, 128])), INVALID),
    (dict(pools=((argus.FP16, 1, 64, None, 4),)), UNSUPPORTED), (dict(pools=((9, 0, 64, None, 4),)), INVALID),
    (dict(pools=((argus.FP16, 0, 64, None, -4),)), INVALID), (dict(pools=((argus.FP16, 0, 64, None, 2 ** 31),)), UNSUPPORTED),
    (dict(pools=((argus.FP16, 0, 72, None, 4),)), INVALID), (dict(pools=((argus.FP16, 0, 64, None, 4), (argus.INT8, 0, 64, None, 4))), INVALID),
    (dict(ws=None), INVALID), (dict(ws=8), INVALID), (dict(ws_bytes=16), WORKSPACE)])
def test_fork_refusals(kw, status):
    assert _fork_status(**kw) == status


def _compact_status(pool=(argus.FP16, 0, 64, None, 40), ws=64, ws_bytes=1 << 40, **kw):
    f = dict(g=argus.geom(2, 2, 64, 16), batch=3, rin=64, rout=128, codec=64, table=64, lens=64, table_out=128, max_pages=4, n_live=64)
    f.update(kw)
    return _lib().argus_compact_pages(ctypes.byref(f["g"]), f["batch"], _pools(pool), f["rin"], f["rout"], f["codec"], f["table"],
                                      f["lens"], f["table_out"], f["max_pages"], f["n_live"], ws, ws_bytes, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=argus.geom(2, 2, 32, 16)), UNSUPPORTED), (dict(batch=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(rin=None), INVALID),
    (dict(rout=64), INVALID), (dict(table_out=64), INVALID), (dict(table=None), INVALID), (dict(n_live=None), INVALID),
    (dict(pool=(argus.INT8, 0, 64, None, 4)), INVALID), (dict(pool=(argus.FP16, 1, 64, None, 4)), UNSUPPORTED),
    (dict(ws=None), INVALID), (dict(ws=8), INVALID), (dict(ws_bytes=16), WORKSPACE)])
def test_compact_refusals(kw, status):
    assert _compact_status(**kw) == status


def test_binding_refuses_tensors_of_another_kind():
    g = argus.geom(4, 2, 64, 16)
    q, i32 = torch.zeros(3, 4, 64, dtype=torch.float16), torch.zeros(8, dtype=torch.int32)
    u8 = torch.zeros(8, dtype=torch.uint8)
    ok = dict(q=q, q_start=i32[:3], pools=[], page_codec=u8, block_table=i32, seq_lens=i32[:2], max_pages=4, softmax_scale=1.0,
              out=torch.empty_like(q))
    argus.extend_args(g, **ok)
    for bad in (dict(q=q[:, :3]), dict(q=q.transpose(0, 1)), dict(q=torch.zeros(3, 4, 128, dtype=torch.float16)[..., ::2]),
                dict(q_start=i32[:3].long()), dict(out=torch.empty(3, 4, 64)), dict(seq_lens=i32[:1]), dict(block_table=i32[:7]),
                dict(page_codec=u8.int()), dict(lse2_out=torch.empty(11)), dict(out=torch.empty(6, 4, 64, dtype=torch.float16)[::2])):
        with pytest.raises(ValueError):
            argus.extend_args(g, **dict(ok, **bad))
    with pytest.raises(ValueError):
        argus.rope_append(g, q, q[:2, :2], q[:, :2], q, i32[:3], i32[:2], i32[:3], torch.zeros(32, dtype=torch.float64), None, u8, i32, 4)


# ---- oracle pins

def test_extend_oracle_is_softmax_attention_row_by_row():
    """16-bit pages: torch's float64 softmax over the gathered keys of every row, and the decode oracle at its last token."""
    rng = np.random.default_rng(1)
    Hkv, G, P, D = 2, 3, 16, 64
    x = rng.standard_normal((9, 2, Hkv, P, D)).astype(np.float16)
    pools = {C.CODEC_FP16: (x.view(np.uint16), None)}
    table = np.array([[3, 8, 1], [0, 5, 7]], np.int32)
    codec = np.zeros((2, 3), np.uint8)
    lens, q_start = [41, 5], [0, 4, 6]
    q = rng.standard_normal((6, Hkv * G, D))
    for causal in (True, False):
        o, lse, bad, *_ = oracle.paged_extend(q, q_start, Hkv, P, pools, codec, table, lens, 0.3, causal)
        assert bad == 0
        for b in range(2):
            kv = torch.from_numpy(x[table[b]].astype(np.float64)).permute(1, 2, 0, 3, 4).reshape(2, Hkv, 3 * P, D)
            n = q_start[b + 1] - q_start[b]
            for i in range(n):
                t = q_start[b] + i
                see = lens[b] - n + i + 1 if causal else lens[b]
                for h in range(Hkv * G):
                    s = 0.3 * kv[0, h // G, :see] @ torch.from_numpy(q[t, h])
                    assert np.allclose(o[t, h], (torch.softmax(s, 0) @ kv[1, h // G, :see]).numpy(), rtol=1e-12, atol=1e-12)
                    assert abs(lse[t, h] * math.log(2) - torch.logsumexp(s, 0).item()) < 1e-12
    one, l1, _ = oracle.paged_decode(q[[3, 5]], Hkv, P, pools, codec, table, lens, 0.3)
    o, lse, *_ = oracle.paged_extend(q, q_start, Hkv, P, pools, codec, table, lens, 0.3, True)
    assert np.allclose(o[[3, 5]], one, rtol=1e-12) and np.allclose(lse[[3, 5]], l1, rtol=1e-12)


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotation_oracle_is_a_complex_product_and_keeps_relative_positions(adjacent):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 2, 64))
    inv = 10000.0 ** (-np.arange(16) / 16)
    pos = rng.integers(-50, 1000, (2, 5))
    axis = np.arange(16) % 2
    y = oracle.rotate(x, pos, inv, axis, adjacent)
    a, b = (np.arange(0, 32, 2), np.arange(1, 32, 2)) if adjacent else (np.arange(16), np.arange(16, 32))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[axis].T * inv)[:, None]
    assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag) and np.array_equal(y[..., 32:], x[..., 32:])
    far = oracle.rotate(x, pos + 2 ** 30, inv, axis, adjacent)
    assert np.allclose((far * np.roll(far, 1, 0))[..., 32:], (x * np.roll(x, 1, 0))[..., 32:])
    d = lambda u: (u[0] * u[0, ::-1])[..., :32].sum()  # noqa: E731  one token's heads among themselves: positions cancel
    assert abs(d(far) - d(x)) < 1e-9


def test_fork_oracle_keeps_counts_equal_to_the_references():
    """After any step, a slot's count is how often it stands in the table plus its outside holders."""
    rng = np.random.default_rng(3)
    B, P, max_pages, n = 12, 16, 10, 400
    table, codec = np.full((B, max_pages), -1, np.int32), np.zeros((B, max_pages), np.uint8)
    lens, refs = np.zeros(B, int), {0: np.zeros(n, int)}
    outside = (rng.random(n) < 0.1).astype(int)
    refs[0] += outside
    for _ in range(30):
        parents = [int(rng.integers(-1, B)) if rng.random() < 0.4 else b for b in range(B)]
        room = [0 if p < 0 else max_pages * P - lens[p] for p in parents]
        new = [int(rng.integers(0, min(20, r) + 1)) for r in room]
        table, codec, lens, refs, copies, st = oracle.fork_pages(parents, new, 0, {0: n}, refs, codec, table, lens, P)
        assert st == 0
        held = outside.copy()
        for b in range(B):
            for j in range((lens[b] + P - 1) // P):
                held[table[b, j]] += 1
        assert np.array_equal(held, refs[0])
        # no two rows write the same page from here
        tails = [table[b, (lens[b] - 1) // P] for b in range(B) if new[b] and lens[b] % P]
        assert len(set(tails)) == len(tails)
        t2, r2, moves, live, bad = oracle.compact_pages(0, refs[0], codec, table, lens, P)
        assert bad == 0 and live == (refs[0] > 0).sum() and np.array_equal(np.sort(r2[:live]), np.sort(refs[0][refs[0] > 0]))
        assert not set(s for s, _ in moves) & set(d for _, d in moves)
