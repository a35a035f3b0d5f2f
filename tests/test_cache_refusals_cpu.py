"""What the binding of the cache operators refuses or holds before any CUDA call."""

import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def pool_of(codec, n_slots=4, hkv=2, page=16, d=64):
    p = argus.Pool.empty(codec, n_slots, hkv, page, d, device="cpu", zero=True)
    return argus.Pool(codec, p.codes, p.meta, n_slots, argus.PLACE_DEVICE)


def extend(**kw):
    f = dict(g=argus.geom(4, 2, 64, 16), q=torch.zeros(3, 4, 64, dtype=torch.float16), q_start=i32(3), pools=[pool_of(argus.FP8_E4M3)],
             page_codec=torch.zeros(2, 4, dtype=torch.uint8), block_table=i32(2, 4), seq_lens=i32(2), max_pages=4, softmax_scale=1.0,
             out=torch.zeros(3, 4, 64, dtype=torch.float16))
    f.update(kw)
    return argus.extend_args(**f)


class _Called(Exception):
    pass


class _Library:
    """Stands for the library: says that the binding let a call through."""

    def __getattr__(self, name):
        def call(*args):
            raise _Called(name)
        return call


@pytest.fixture
def no_library(monkeypatch):
    monkeypatch.setattr(argus, "lib", lambda: _Library())
    monkeypatch.setattr(argus, "_stream_of", lambda device, stream: None)


def rope(**kw):
    f = dict(g=argus.geom(4, 2, 64, 16), q=torch.zeros(3, 4, 64, dtype=torch.float16), k=torch.zeros(3, 2, 64, dtype=torch.float16),
             v=torch.zeros(3, 2, 64, dtype=torch.float16), q_out=torch.zeros(3, 4, 64, dtype=torch.float16), q_start=i32(3), seq_lens=i32(2),
             positions=i32(1, 3), inv_freq=torch.zeros(32, dtype=torch.float64), pool=pool_of(argus.FP16),
             page_codec=torch.zeros(2, 4, dtype=torch.uint8), block_table=i32(2, 4), max_pages=4)
    f.update(kw)
    argus.rope_append(**f)


def tokens_over_each_other(heads, step):
    return torch.zeros(step * 2 + heads * 64, dtype=torch.float16).as_strided((3, heads, 64), (step, 64, 1))


@pytest.mark.parametrize("step", [0, 64, 248])
def test_tokens_that_share_memory_are_refused(no_library, step):
    """A tensor broadcast over its tokens holds one token; its stride of 0 must not reach the library, where 0 means dense."""
    with pytest.raises(ValueError, match="overlap"):
        extend(q=tokens_over_each_other(4, step))
    for name, heads in (("q", 4), ("k", 2), ("v", 2), ("q_out", 4)):
        with pytest.raises(ValueError, match="overlap"):
            rope(**{name: tokens_over_each_other(heads, min(step, 120))})


def test_single_and_strided_tokens_are_taken(no_library):
    with pytest.raises(_Called):
        rope()
    wide = torch.zeros(3, 8, 64, dtype=torch.float16)
    with pytest.raises(_Called):
        rope(q=wide[:, :4], k=wide[:, 4:6], v=wide[:, 6:])
    assert extend(q=wide[:, 2:6]).q_stride == 512 and extend().q_stride == 256
    # one token, however its tensor was made, is dense
    one = torch.zeros(1, 4, 64, dtype=torch.float16)
    for q in (one, one[0].expand(1, 4, 64), tokens_over_each_other(4, 0)[:1]):
        assert extend(q=q, q_start=i32(2), seq_lens=i32(1), out=torch.zeros(1, 4, 64, dtype=torch.float16)).q_stride == 256


def fork(pool, **kw):
    table, codec = i32(2, 4), torch.zeros(2, 4, dtype=torch.uint8)
    argus.fork_pages(kw.get("g", argus.geom(4, 2, 64, 16)), i32(2), i32(2), argus.FP16, [pool_of(argus.FP16), pool],
                     [i32(4), i32(max(pool.n_slots, 0))], [i32(4), i32(max(pool.n_slots, 0))], codec, table, i32(2), codec.clone(),
                     table.clone(), i32(2), 4, torch.zeros(64, dtype=torch.uint8))


def compact(pool, **kw):
    table, codec, ref = i32(2, 4), torch.zeros(2, 4, dtype=torch.uint8), i32(max(pool.n_slots, 0))
    argus.compact_pages(kw.get("g", argus.geom(4, 2, 64, 16)), pool, ref, ref.clone(), codec, table, i32(2), table.clone(), 4, i32(1),
                        torch.zeros(64, dtype=torch.uint8))


def takes(call, *args, **kw):
    with pytest.raises(_Called):
        call(*args, **kw)


ALL = [argus.FP16, argus.BF16, argus.FP8_E4M3, argus.INT8, argus.INT4_G32, argus.INT2_G32, argus.INT1_G32]


@pytest.mark.parametrize("codec", ALL)
def test_pools_that_do_not_hold_their_pages_are_refused(no_library, codec):
    """Slots are checked against n_slots alone on the device: n_slots pages of this geometry have to be there."""
    whole = pool_of(codec)
    calls = [fork, compact] if codec != argus.FP16 else [compact]
    if codec <= argus.INT8:
        calls.append(lambda pool, **kw: extend(pools=[pool], **kw))
    if codec == argus.FP16:
        calls.append(lambda pool, **kw: rope(pool=pool, **kw))

    def like(**kw):
        f = dict(codes=whole.codes, meta=whole.meta, n_slots=4)
        f.update(kw)
        return argus.Pool(codec, f["codes"], f["meta"], f["n_slots"], argus.PLACE_DEVICE)

    wide = torch.zeros(whole.codes.shape[:-1] + (2 * whole.codes.shape[-1],), dtype=whole.codes.dtype)
    bad = [dict(n_slots=5), dict(codes=whole.codes[:3]), dict(codes=wide[..., :whole.codes.shape[-1]]), dict(codes=whole.codes.transpose(1, 2)),
           dict(codes=whole.codes[:1].expand(whole.codes.shape)), dict(codes=whole.codes.double()),
           dict(codes=torch.zeros(whole.codes.shape, dtype=torch.float8_e5m2 if codec >= argus.FP8_E4M3 else torch.float32))]
    if whole.meta is not None:
        bad += [dict(meta=whole.meta[:3]), dict(meta=whole.meta.double()), dict(meta=whole.meta.bfloat16()),
                dict(meta=whole.meta[:1].expand(whole.meta.shape)), dict(meta=whole.meta.transpose(1, 2)),
                dict(meta=whole.meta.half() if codec < argus.INT4_G32 else whole.meta.float())]
    for call in calls:
        for kw in bad:
            with pytest.raises(ValueError, match="pool"):
                call(like(**kw))
        for g in (argus.geom(8, 4, 64, 16), argus.geom(4, 2, 128, 16), argus.geom(4, 2, 64, 32)):
            with pytest.raises(ValueError, match="pool"):
                call(whole, g=g)


def test_pools_of_other_shapes_and_raw_types_are_taken(no_library):
    """A pool may be larger, flat, of the codes' own float type, or hold its bits as integers."""
    p = pool_of(argus.FP8_E4M3, n_slots=6)
    for codes in (p.codes, p.codes.flatten(), p.codes.view(torch.float8_e4m3fn), p.codes.view(torch.int8), p.codes.view(torch.int32)):
        for n in (0, 4, 6):
            extend(pools=[argus.Pool(argus.FP8_E4M3, codes, p.meta.flatten(), n, argus.PLACE_DEVICE)])
    takes(compact, argus.Pool(argus.BF16, pool_of(argus.BF16).codes.view(torch.int16), None, 4, argus.PLACE_DEVICE))
    extend(pools=[argus.Pool(argus.FP8_E4M3, None, None, 0, argus.PLACE_DEVICE)])
    for codec in ALL[1:]:
        takes(fork, pool_of(codec))
        takes(compact, pool_of(codec))
    takes(rope, pool=pool_of(argus.FP16))


def test_extend_args_keep_the_pools_alive():
    """The caller's list of pools, and the pools' own tensors, may change between building the arguments and the call."""
    import gc
    import weakref
    pools = [pool_of(argus.FP8_E4M3), pool_of(argus.INT8)]
    held = [weakref.ref(t) for p in pools for t in (p.codes, p.meta)]
    args = extend(pools=pools)
    pools[1].codes = pools[1].meta = None
    pools.clear()
    gc.collect()
    assert all(r() is not None for r in held)
    del args
    gc.collect()
    assert all(r() is None for r in held)
