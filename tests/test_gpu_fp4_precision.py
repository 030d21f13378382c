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


@pytest.mark.parametrize("S,most,long", [(6000, 20, 5000), (65535, 3, 3000), (12345, 1, 0)])
def test_thousands_of_sequences(S, most, long):
    """More sequences than the CTAs' threads count one by one; some empty, a long one near the end."""
    H, Hk, bs = 2, 1, 16
    g = torch.Generator().manual_seed(S)
    lens = torch.randint(0, most + 1, (S,), generator=g)
    lens[-1] = most
    if long:
        lens[S - 37] = long
    tables, NB = F.shuffled_tables(lens.tolist(), bs, g, extra=0)
    cache = F.U.random_cache4(NB, Hk, bs, 1.0, g, wild=True)
    # group scales of 2^-3 to 1, so that the logits of a sequence lie within reach of one another
    cache[..., 128 * bs:] = torch.randint(0x20, 0x38, cache[..., 128 * bs:].shape, generator=g, dtype=torch.uint8)
    q = torch.randn(S, H, 128, generator=g).to(torch.bfloat16)
    scale, ks, vs = 0.125, 0.25, 0.5
    got = pda.decode_fp4(q.to(DEV), cache.to(DEV), tables.to(DEV), i32(lens), scale, ks, vs).double().cpu()
    want, mean, top = F.decode_by_length(q, cache, tables, lens, bs, scale, ks, vs)
    # f16 weights 2^-11; logits: 128 products in binary32, 2^-16 of scale ks sum |q k|, twice (numerator and sum), with
    # |k| < 6 and sum |q| < 160, so 2^-10; sums of 5000 / 16 steps 2^-13; small weights; the output
    assert float(q.double().abs().sum(-1).max()) < 160
    tol = mean * (2.0 ** -11 + 2.0 ** -9) + top * 2.0 ** -32 + want.abs() * 2.0 ** -8
    err = (got - want).abs()
    assert (err <= tol).all(), (int((err > tol).sum()), float((err / tol.clamp(min=1e-30)).max()))
    assert (got[lens == 0] == 0).all()
    assert pda.query_device_status() == 0


@pytest.mark.parametrize("size", [0, 4, 8, 12, 16, 18])
@pytest.mark.parametrize("lens,H,Hk,bs,alone", [([64, 33, 7, 0], 8, 4, 16, True), ([300, 5], 8, 2, 128, False), ([5000], 16, 2, 16, False),
                                                ([2500, 40], 12, 4, 32, False)])
def test_logits_of_any_size(size, lens, H, Hk, bs, alone):
    """Logits of about 2^size that differ by 12 at most, all exact in binary32, so that nothing but the weights is rounded. Where one
    warp sees a whole head (`alone`) that holds at every size; where parts are merged, their references round too, and
    weights are as precise as the calls promise (size * 2^-22)."""
    g = torch.Generator().manual_seed(size + bs)
    tables, NB = F.shuffled_tables(lens, bs, g, extra=0)
    cache = torch.zeros(NB, Hk, 144 * bs, dtype=torch.uint8)
    grid = torch.from_numpy(F.U.E2M1)
    scale, ks, vs = 0.5, 0.25, 0.5
    q = torch.zeros(len(lens), H, 128, dtype=torch.bfloat16)
    q[..., 0] = 2.0 ** (size - 7)
    q[..., 16:32] = 1.0
    key, val = [], []
    for i, n in enumerate(lens):
        pos = torch.arange(n)
        slots = tables[i, pos // bs].long() * bs + pos % bs
        k = torch.zeros(n, Hk, 128, dtype=torch.float64)
        k[..., 0] = 4
        k[..., 16:32] = grid[torch.randint(0, 8, (n, Hk, 16), generator=g)] * (1 - 2 * torch.randint(0, 2, (n, Hk, 16), generator=g))
        s = torch.ones(n, Hk, 8, dtype=torch.float64)
        s[..., 0] = 256
        F.write_rows(cache, bs, 0, slots, k, s)
        v = grid[torch.randint(0, 8, (n, Hk, 128), generator=g)] * (1 - 2 * torch.randint(0, 2, (n, Hk, 128), generator=g))
        F.write_rows(cache, bs, 1, slots, v, torch.ones(n, Hk, 8))
        key.append(k[..., 16:32].sum(-1) * scale * ks)              # the rest is the same for every token
        val.append(v * vs)
    got = pda.decode_fp4(q.to(DEV), cache.to(DEV), tables.to(DEV), i32(lens), scale, ks, vs).double().cpu()
    # the weights' f16 (2^-11), the exponents' products of up to 40 in binary32 and the exponential (2^-17 together), sums of up
    # to 5000 / 16 steps (2^-13); the promised precision, in numerator and sum
    part = 2.0 ** -11 + 2.0 ** -12 + (0 if alone else 2 * 2.0 ** (size - 22))
    for i, n in enumerate(lens):
        for h in range(H):
            if n == 0:
                assert (got[i, h] == 0).all()
                continue
            w = torch.softmax(key[i][:, h // (H // Hk)], 0)
            v = val[i][:, h // (H // Hk)]
            want = w @ v
            tol = (w @ v.abs()) * part + 2.0 ** -32 * n * 3 + want.abs() * 2.0 ** -8
            assert ((got[i, h] - want).abs() <= tol).all(), (i, h, float(((got[i, h] - want).abs() / tol).max()))
    assert pda.query_device_status() == 0


@pytest.mark.parametrize("H,Hk,bs,lens,window,with_sinks", [(32, 8, 16, [3, 0, 700, 64], 0, False), (6, 2, 32, [1, 129, 2000], 0, True),
                                                            (8, 1, 128, [5, 3000], 100, False), (21, 3, 48, [47, 600, 0], 333, True),
                                                            (4, 4, 16, [30, 30], 0, True)])
def test_e4m3_output_of_every_path(H, Hk, bs, lens, window, with_sinks):
    """e4m3 rows written by one warp, merged in a CTA, and joined."""
    from tests.test_gpu_decode_fp4 import KS, VS, Batch
    b = Batch(lens, H, Hk, bs, seed=H + bs)
    kw = dict(window=window, sinks=torch.randn(H, generator=torch.Generator().manual_seed(7)) if with_sinks else None)
    s = 0.003
    got = b.run(output_scale=s, **kw).cpu()
    assert got.dtype == torch.float8_e4m3fn
    want, tol = F.U.decode64(b.q, b.cache, b.tables, b.lens, bs, b.scale, KS, VS, **kw)
    want, far = want / s, tol / s
    # the e4m3 rounding is monotonic: half a step (2^-4, 2^-10 below its normals) of what the kernel rounds
    limit = far + (want.abs() + far) * 2.0 ** -4 + 2.0 ** -10
    assert ((got.double() - want.clamp(-448, 448)).abs() <= limit).all()
    assert pda.query_device_status() == 0
