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
