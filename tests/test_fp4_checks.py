"""The checks of the 4-bit decode's long and far contexts tell mistakes, on the CPU: each is planted in the plain form."""

import pytest
import torch

from tests import fp4_util as F


def f16(w):
    return w.float().half().double()


def test_far_token_tells_small_weights():
    """Weights held with seven binary places below one agree; held as f16 relative to the largest they do not, nor does a
    token that is left out."""
    c = F.FarToken(513, 40, 8, 2, 32, seed=1)
    want, tol = c.plain()
    got, _ = c.plain(weights=lambda w: f16(w * 128) / 128)
    assert ((got - want).abs() <= tol).all()
    got, _ = c.plain(weights=f16)
    assert ((got - want).abs() > tol).any()
    sinks = torch.linspace(-5, 25, 8)
    want, tol = c.plain(sinks=sinks)
    got, _ = c.plain(sinks=sinks + 7 * 0.6931)                      # a sink in another unit than the weights
    assert ((got - want).abs() > tol).any()


@pytest.mark.parametrize("lens,H,Hk,bs,window", F.MARKED)
def test_marks_tell_every_page(lens, H, Hk, bs, window):
    c = F.MarkedPages(lens, H, Hk, bs, cache=False)
    for i, n in enumerate(lens[:5]):
        lo = max(0, n - window) if window else 0
        first, pages = lo // bs, -(-n // bs)
        want = c.plain(i, window)
        assert c.agrees(want, want).all()
        if pages - first < 2:
            continue
        for j in {first, first + 1, first + 255, first + 256, (first + pages) // 2, pages - 2, pages - 1} & set(range(first, pages)):
            if min(n, (j + 1) * bs) - max(lo, j * bs) < bs / 2:     # a sliver of a page
                continue
            for kw in (dict(drop=[j]), dict(twice=[j])):
                assert not c.agrees(c.plain(i, window, **kw), want).all(1).any(), (i, j, kw)
        # a run of pages, such as a piece of the work
        for a in range(first, pages - 9, max(1, (pages - first) // 7)):
            assert not c.agrees(c.plain(i, window, drop=range(a, a + 9)), want).all(1).any()
