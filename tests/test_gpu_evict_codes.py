"""argus_evict_tokens into 8-bit pages, every byte against the oracle's encoders (which argus_quantize_pages equals bit for
bit): pages whose scale is subnormal, and the sign of zero."""

import numpy as np
import pytest
import torch

import mixed_precision_paged_argus_gb300.argus as argus
from mixed_precision_paged_argus_gb300 import workloads as W
import oracle
from oracle import codecs as C
from test_gpu_evict import call, weights
from test_gpu_extend import F8, I8, make

pytestmark = pytest.mark.gpu
UNIT = 2.0 ** -149                                       # fp32's smallest step


def evicted(c, to, budget=130):
    """The call's pages and the oracle's, as bytes."""
    w = weights(c, 1)
    e = call(c, w, budget, 4, 30, to)
    codes, meta = C.alloc_pool(to, e.n_slots, c.Hkv, c.P, c.D)
    codes.view(np.uint8)[...], meta[...] = 0x3C, 7.0
    oracle.evict_tokens(c.Hkv, c.P, c.D, c.opools, c.page_codec, c.table, c.lens, w, budget, 4, 30, to, codes, meta, e.table, e.w.shape[2])
    assert np.array_equal(e.dst.meta.cpu().numpy(), meta)
    return e, e.dst.codes.cpu().view(torch.uint8).numpy(), codes.view(np.uint8)


@pytest.mark.parametrize("P", [16, 64, 160])
@pytest.mark.parametrize("codecs", [[F8], [I8], [F8, I8], [I8, W.INT4_G32]])
def test_int8_codes_of_subnormal_scales(codecs, P):
    """Where top / 127 is a few units of 2^-149 its rounding takes x / scale far past 127, which is where a code ends."""
    c = make(4, 3, 64, P, [900, 333, 40], [1] * 3, codecs, W.FP16, seed=174 + P)
    rng = np.random.default_rng(11)
    for pool in c.pools:
        if pool.codec in (F8, I8):
            # scales of 1 to 2^17 units, many of few; in every unit some value of 100 units, so that none has the scale 0
            codes, meta = c.opools[pool.codec]
            meta[...] = np.rint(2.0 ** rng.uniform(0, 17 if P == 16 else 3, meta.shape)) * UNIT
            codes.view(np.uint8)[..., 5] = {F8: 0x7E, I8: 100}[pool.codec]
            pool.codes.view(torch.uint8).copy_(torch.from_numpy(codes.view(np.uint8)))
            pool.meta.copy_(torch.from_numpy(meta))
    if W.INT4_G32 in codecs:                             # rows of zeros beside them
        for pool in c.pools:
            if pool.codec == W.INT4_G32:
                pool.meta.zero_()
                c.opools[pool.codec][1][...] = 0
    e, got, want = evicted(c, I8)
    scales = e.dst.meta[torch.from_numpy(e.table).flatten().long()]
    assert (scales < 100 * UNIT).any()
    assert np.array_equal(got, want)


@pytest.mark.parametrize("P", [16, 160])
@pytest.mark.parametrize("codecs", [[F8], [W.BF16], [W.BF16, F8], [W.BF16, I8]])
def test_fp8_codes_keep_the_sign_of_zero(codecs, P):
    c = make(4, 2, 128, P, [500, 90], [1, 1], codecs, W.BF16, seed=180 + P)
    rng = np.random.default_rng(12)
    for pool in c.pools:
        if pool.codec == I8:
            continue
        codes, _ = c.opools[pool.codec]
        zero = rng.random(codes.shape) < 0.3
        codes[zero] = rng.choice([0, 0x80 if pool.codec == F8 else 0x8000], int(zero.sum()))
        pool.codes.view(torch.uint8).copy_(torch.from_numpy(codes.view(np.uint8).reshape(pool.codes.view(torch.uint8).shape)))
    _, got, want = evicted(c, F8)
    assert (want == 0x80).any() and (want == 0).any()
    assert np.array_equal(got, want)


@pytest.mark.parametrize("to", [F8, I8])
def test_codes_are_those_of_demotion(to):
    """Evicted to 16 bits and demoted, or evicted to 8 bits: the same bytes."""
    c = make(4, 2, 64, 16, [400, 700], [1, 1], [W.BF16], W.BF16, seed=190)
    pool = c.pools[0]
    pool.codes[torch.rand(pool.codes.shape, device=pool.codes.device) < 0.2] = -0.0
    w = weights(c, 2)
    wide = call(c, w, 160, 4, 30, W.BF16)
    direct = call(c, w, 160, 4, 30, to)
    demoted = argus.Pool.empty(to, wide.n_slots, c.Hkv, c.P, c.D, device=pool.codes.device, zero=True)
    slots = torch.from_numpy(wide.table.flatten()).to(pool.codes.device)
    argus.quantize_pages(c.g, W.BF16, wide.dst.codes, wide.n_slots, slots, demoted, slots, slots.numel())
    at = slots.long()
    assert torch.equal(demoted.codes.view(torch.uint8)[at], direct.dst.codes.view(torch.uint8)[at])
    assert torch.equal(demoted.meta[at], direct.dst.meta[at])
