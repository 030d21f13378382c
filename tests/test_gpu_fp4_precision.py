"""Decode attention over the 4-bit cache where single weights and single pages decide (inputs, tolerances: fp4_util)."""

import pytest
import torch

import paged_kv_decode_pda_gb300 as pda
from tests import fp4_util as F

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("H,Hk,bs", [(16, 8, 16), (32, 4, 16), (6, 2, 32), (8, 1, 128), (3, 3, 48)])
@pytest.mark.parametrize("with_sinks", [False, True])
def test_small_weights(H, Hk, bs, with_sinks):
    """A token up to 2^33 times as heavy as the others, whose V is zero: the others' weights alone make the output."""
    c = F.FarToken(513, 240, H, Hk, bs, seed=H + bs)
    sinks = torch.linspace(-5, 25, H) if with_sinks else None
    got = pda.decode_fp4(c.q.to(DEV), c.cache.to(DEV), c.tables.to(DEV).expand(c.S, -1).contiguous(), i32([c.n] * c.S), c.scale, c.ks,
                         c.vs, sinks=None if sinks is None else sinks.to(DEV)).double().cpu()
    want, tol = c.plain(sinks=sinks)
    err = (got - want).abs()
    assert (err <= tol).all(), (int((err > tol).sum()), float((err / tol).max()))
    assert pda.query_device_status() == 0


@pytest.mark.parametrize("lens,H,Hk,bs,window", F.MARKED)
def test_every_page_counts(lens, H, Hk, bs, window):
    """Long units over many CTAs, up to all of them: equal weights over distinct pages, each seen in a dim of its own set."""
    c = F.MarkedPages(lens, H, Hk, bs, seed=len(lens) + bs)
    dev = c.q.to(DEV), c.cache.to(DEV), c.tables.to(DEV), i32(lens)
    for _ in range(3):
        got = pda.decode_fp4(*dev, 0.1, 1.0, c.vs, window=window).double().cpu()
        for i in range(len(lens)):
            want = c.plain(i, window).repeat_interleave(H // Hk, 0)
            assert c.agrees(got[i], want).all(), (i, torch.nonzero(~c.agrees(got[i], want))[:5].tolist())
    assert pda.query_device_status() == 0
