"""The quantising cache writers and the readers against their plain forms, byte for byte."""

import numpy as np
import pytest
import torch

import paged_kv_decode_pda_gb300 as pda
from tests import lowbits_util as U

pytestmark = pytest.mark.gpu
DEV = "cuda"
MIN = 2.0 ** -20


def gen(seed):
    return torch.Generator().manual_seed(seed)


def special(x, seed):
    """Rows with the values that are easily got wrong: zeros, a lone value, infinities, NaN, tiny, huge, ties."""
    T = x.shape[0]
    x[0 % T] = 0.0
    if T > 1:
        x[1, :, :] = 0.0
        x[1, :, 77] = -3.0
    if T > 2:
        x[2, :, 5] = float("inf")
        x[2, :, 100] = -float("inf")
    if T > 3:
        x[3, :, 40] = float("nan")
    if T > 4:
        x[4] = x[4] * 2.0 ** -120
    if T > 5:
        x[5] = x[5] * 2.0 ** 100
    if T > 6:
        x[6] = torch.arange(-64, 64).to(torch.bfloat16) / 8     # eighths: ties wherever the scale is a power of two
    if T > 7:
        x[7, :, :16] = 0.0
        x[7, :, 3] = float("inf")                               # an infinity among zeros
    return x


def tokens(T, Hk, seed, layout):
    """(key, value) [T, Hk, 128] bf16 on the GPU: contiguous, views of a packed projection, or off the 16-byte grid."""
    g = gen(seed)
    loud = (torch.randn(T, 1, 1, generator=g)).exp()
    kv = [special((torch.randn(T, Hk, 128, generator=g) * loud).to(torch.bfloat16), seed) for _ in range(2)]
    if layout == "plain":
        return [x.to(DEV) for x in kv]
    if layout == "packed":
        buf = torch.zeros(T, 4 * Hk * 128, dtype=torch.bfloat16, device=DEV)
        k, v = buf[:, Hk * 128:2 * Hk * 128].view(T, Hk, 128), buf[:, 3 * Hk * 128:].view(T, Hk, 128)
    elif layout == "heads_first":
        buf = torch.zeros(2, Hk, T, 128, dtype=torch.bfloat16, device=DEV)
        k, v = buf[0].transpose(0, 1), buf[1].transpose(0, 1)
    else:                                                       # rows 131 apart, from an odd element on
        buf = torch.zeros(2 * T * Hk * 131 + 1, dtype=torch.bfloat16, device=DEV)
        k = buf[1:1 + T * Hk * 131].view(T, Hk, 131)[..., :128]
        v = buf[1 + T * Hk * 131:].view(T, Hk, 131)[..., 2:130]
    k.copy_(kv[0])
    v.copy_(kv[1])
    return [k, v]


def slots_for(kind, T, NB, bs, seed):
    g = gen(seed)
    if kind == "scattered":
        s = torch.randperm(NB * bs, generator=g)[:T]
        s[torch.rand(T, generator=g) < 0.15] = -1
    elif kind == "blocks":
        blocks = torch.randperm(NB, generator=g)[:-(-T // bs)]
        t = torch.arange(T)
        s = blocks[t // bs] * bs + t % bs
    else:                                                       # a run that starts inside a block, in an ascending pool
        s = torch.arange(T) + 5
    return s


WRITES = [(1, 1, 16, "scattered", "plain"), (7, 3, 16, "scattered", "odd"), (16, 8, 16, "blocks", "plain"),
          (33, 2, 32, "blocks", "packed"), (50, 1, 48, "run", "heads_first"), (130, 8, 64, "run", "packed"),
          (257, 4, 128, "blocks", "odd"), (300, 2, 16, "scattered", "packed"), (96, 5, 16, "run", "plain")]


@pytest.mark.parametrize("T,Hk,bs,kind,layout", WRITES)
@pytest.mark.parametrize("least", [MIN, 0.5])
def test_write_slot_scales(T, Hk, bs, kind, layout, least):
    NB = -(-(T + 5) // bs) + 2
    k, v = tokens(T, Hk, T + bs, layout)
    slots = slots_for(kind, T, NB, bs, T)
    g = gen(3)
    kc = torch.randint(0, 256, (NB, Hk, 8, bs, 16), generator=g, dtype=torch.uint8)
    vc = torch.randint(0, 256, (NB, Hk, 128, bs), generator=g, dtype=torch.uint8)
    ks, vs = (torch.rand(NB, Hk, bs, generator=g) for _ in range(2))
    dev = [x.to(DEV) for x in (kc, vc, ks, vs)]
    pda.reshape_and_cache_slot_scales(k, v, *dev, slots.to(DEV), min_scale=least)
    ck, sk = U.quantize_rows8(k.cpu(), least)
    cv, sv = U.quantize_rows8(v.cpu(), least)
    for t, s in enumerate(slots.tolist()):
        if s < 0:
            continue
        b, o = s // bs, s % bs
        kc[b, :, :, o] = ck[t].view(Hk, 8, 16)
        vc[b, :, :, o] = cv[t]
        ks[b, :, o], vs[b, :, o] = sk[t], sv[t]
    # a NaN's sign is free
    for got, want in zip(dev[:2], (kc, vc)):
        got = got.cpu()
        same = (got == want) | (((got & 0x7F) == 0x7F) & ((want & 0x7F) == 0x7F))
        assert same.all(), torch.nonzero(~same)[:5]
    assert torch.equal(dev[2].cpu(), ks) and torch.equal(dev[3].cpu(), vs)
    assert pda.query_device_status() == 0


@pytest.mark.parametrize("T,Hk,bs,kind,layout", WRITES)
@pytest.mark.parametrize("ks,vs", [(0.0043, 0.0039), (2.0 ** -8, 2.0 ** -9), (1e-20, 1e20)])
def test_write_fp4(T, Hk, bs, kind, layout, ks, vs):
    NB = -(-(T + 5) // bs) + 2
    k, v = tokens(T, Hk, T + bs, layout)
    slots = slots_for(kind, T, NB, bs, T)
    want = torch.randint(0, 256, pda.fp4_cache_shape(NB, Hk, bs), generator=gen(4), dtype=torch.uint8)
    got = want.to(DEV)
    pda.reshape_and_cache_fp4(k, v, got, slots.to(DEV), ks, vs)
    for kind4, x, g in ((0, k, ks), (1, v, vs)):
        codes, scales = U.quantize_rows4(x.cpu(), g)
        U.write4(want, bs, kind4, slots, codes, scales)
    got = got.cpu()
    if not torch.equal(got, want):
        # the codes of a group that holds a NaN are free: compare what is read
        every = torch.arange(NB * bs)
        for kind4 in range(2):
            a, b = (U.read4(c, bs, kind4, every // bs, every % bs, 1.0)[0] for c in (got, want))
            assert torch.equal(torch.nan_to_num(a, nan=-1.0), torch.nan_to_num(b, nan=-1.0))
        assert torch.equal(got[..., 128 * bs:], want[..., 128 * bs:])
    assert pda.query_device_status() == 0


def every_quotient(width, binades):
    """Rows [., 128] bf16: each group of `width` dims holds a largest value (all 128 significands in turn) and others of every
    significand in the `binades` binades below it, of both signs."""
    sig = torch.arange(128, dtype=torch.float64) / 128 + 1
    x = (sig[None] * 2.0 ** -torch.arange(1, binades + 1, dtype=torch.float64)[:, None]).flatten()
    x = torch.cat([sig, x])                                     # of the largest's own binade too, those that are not larger
    x = x * (1 - 2 * (torch.arange(len(x)) % 3 == 0).double())
    rows = []
    for a in sig:
        y = x[x.abs() <= a]
        y = torch.cat([y, y.new_zeros(-len(y) % (width - 1))]).view(-1, width - 1)
        rows.append(torch.cat([a.expand(len(y), 1), y], 1))
    rows = torch.cat(rows).flatten()
    return torch.cat([rows, rows.new_zeros(-len(rows) % 128)]).view(-1, 128).to(torch.bfloat16)


@pytest.mark.parametrize("heads", [1, 2])
def test_every_quotient_slot_scales(heads):
    """Every pair of significands (a row's largest, another value) down to codes of zero, both kernels: each code the nearest."""
    x = every_quotient(128, 20)[:, None].expand(-1, heads, -1).contiguous()
    T, bs = x.shape[0], 16
    assert (T * heads > 4096) == (heads == 2)
    NB = -(-T // bs)
    dev = [torch.zeros(NB, heads, 8, bs, 16, dtype=torch.uint8, device=DEV), torch.zeros(NB, heads, 128, bs, dtype=torch.uint8, device=DEV),
           torch.zeros(NB, heads, bs, device=DEV), torch.zeros(NB, heads, bs, device=DEV)]
    key, value = x.to(DEV), (x * -2.0 ** 30).to(DEV)
    pda.reshape_and_cache_slot_scales(key, value, *dev, torch.arange(T, device=DEV))
    kc, vc, ks, vs = (t.cpu() for t in dev)
    t = torch.arange(T)
    for cache, table, rows in ((kc[t // bs, :, :, t % bs].reshape(T, heads, 128), ks, key), (vc[t // bs, :, :, t % bs], vs, value)):
        codes, scales = U.quantize_rows8(rows.cpu(), MIN)
        assert torch.equal(cache, codes) and torch.equal(table[t // bs, :, t % bs], scales)


@pytest.mark.parametrize("g", [2.0 ** -8, 0.0043, 7.0 / 1024, 1.0 / 3])
def test_every_quotient_fp4(g):
    """Every pair of significands (a group's largest, another value) down to codes of zero; groups of several magnitudes."""
    x = every_quotient(16, 5)
    x = torch.cat([x * f for f in (2.0 ** -9, 1.0, 2.0 ** 3)])[:, None].contiguous()
    T, bs = x.shape[0], 16
    NB = -(-T // bs)
    want = torch.zeros(pda.fp4_cache_shape(NB, 1, bs), dtype=torch.uint8)
    got = want.to(DEV)
    value = -x.flip(0)
    slots = torch.arange(T)
    pda.reshape_and_cache_fp4(x.to(DEV), value.to(DEV), got, slots.to(DEV), g, g)
    for kind, rows in ((0, x), (1, value)):
        U.write4(want, bs, kind, slots, *U.quantize_rows4(rows, g))
    assert torch.equal(got.cpu(), want)


# past 4096 rows (tiles of 16 tokens), and past 9728 (four heads of a token to a warp)
MANY = [(600, 8, 16, "blocks", "plain"), (1100, 9, 32, "run", "packed"), (530, 9, 64, "scattered", "odd"),
        (2100, 2, 128, "blocks", "heads_first"), (4105, 1, 48, "run", "plain"), (1300, 10, 16, "scattered", "odd"),
        (2600, 5, 16, "run", "heads_first"), (9800, 1, 64, "scattered", "packed")]


@pytest.mark.parametrize("T,Hk,bs,kind,layout", MANY)
def test_write_many_slot_scales(T, Hk, bs, kind, layout):
    test_write_slot_scales(T, Hk, bs, kind, layout, MIN)


@pytest.mark.parametrize("T,Hk,bs,kind,layout", MANY)
def test_write_many_fp4(T, Hk, bs, kind, layout):
    test_write_fp4(T, Hk, bs, kind, layout, 0.0043, 0.0039)


def test_write_many_in_any_order():
    """Slots in descending order, and runs that change blocks inside a tile: every way a tile's tokens fall into groups of 16 slots."""
    T, Hk, bs = 600, 8, 32
    NB = T // bs + 3
    k, v = tokens(T, Hk, 50, "plain")
    g = gen(51)
    runs = torch.randperm(T // 5, generator=g)
    for slots in (T + 20 - torch.arange(T), (runs[:, None] * 5 + torch.arange(5)).flatten() + 3):
        kc, vc = (torch.zeros(NB, Hk, *s, dtype=torch.uint8, device=DEV) for s in ((8, bs, 16), (128, bs)))
        ks, vs = (torch.zeros(NB, Hk, bs, device=DEV) for _ in range(2))
        pda.reshape_and_cache_slot_scales(k, v, kc, vc, ks, vs, slots.to(DEV))
        b, o = slots // bs, slots % bs
        for x, cache, scales in ((k, kc.cpu().permute(0, 3, 1, 2, 4).reshape(NB, bs, Hk, 128), ks),
                                 (v, vc.cpu().permute(0, 3, 1, 2), vs)):
            codes, s = U.quantize_rows8(x.cpu(), MIN)
            got = cache[b, o]
            assert ((got == codes) | (((got & 0x7F) == 0x7F) & ((codes & 0x7F) == 0x7F))).all()
            assert torch.equal(scales.cpu().permute(0, 2, 1)[b, o], s)
            assert int((scales != 0).sum()) == T * Hk


def test_write_many_with_repeated_slots():
    """Rows of one content at one slot leave that content, also several in a tile; the neighbours stay whole."""
    T, Hk, bs = 600, 8, 16
    k, v = tokens(T, Hk, 52, "plain")
    slots = torch.arange(T)
    for a, b in ((17, 18), (20, 31), (21, 31), (100, 500), (599, 0), (64, 79), (65, 79), (66, 79)):
        k[a], v[a], slots[a] = k[b], v[b], slots[b]
    NB = -(-T // bs)
    kc, vc = (torch.zeros(NB, Hk, *s, dtype=torch.uint8, device=DEV) for s in ((8, bs, 16), (128, bs)))
    ks, vs = (torch.zeros(NB, Hk, bs, device=DEV) for _ in range(2))
    pda.reshape_and_cache_slot_scales(k, v, kc, vc, ks, vs, slots.to(DEV))
    for x, cache, scales in ((k, kc.cpu().permute(0, 3, 1, 2, 4).reshape(NB, bs, Hk, 128), ks), (v, vc.cpu().permute(0, 3, 1, 2), vs)):
        codes, s = U.quantize_rows8(x.cpu(), MIN)
        got = cache[slots // bs, slots % bs]
        assert ((got == codes) | (((got & 0x7F) == 0x7F) & ((codes & 0x7F) == 0x7F))).all()
        assert torch.equal(scales.cpu().permute(0, 2, 1)[slots // bs, slots % bs], s)
    assert int((ks.permute(0, 2, 1).reshape(-1, Hk)[[17, 20, 21, 100, 599, 64, 65, 66]] != 0).sum()) == 0


def test_writes_skip_slots_past_the_pool():
    k, v = tokens(3, 2, 1, "plain")
    slots = torch.tensor([5, 16 * 2, -1], device=DEV)
    cache = torch.zeros(pda.fp4_cache_shape(2, 2, 16), dtype=torch.uint8, device=DEV)
    pda.reshape_and_cache_fp4(k, v, cache, slots, 0.01, 0.01)
    assert pda.query_device_status() == 16
    kc, vc = (torch.zeros(2, 2, *s, dtype=torch.uint8, device=DEV) for s in ((8, 16, 16), (128, 16)))
    ks, vs = (torch.zeros(2, 2, 16, device=DEV) for _ in range(2))
    pda.reshape_and_cache_slot_scales(k, v, kc, vc, ks, vs, slots)
    assert pda.query_device_status() == 16
    assert int((ks != 0).sum()) == 2 and int((cache.view(4, -1)[:, 128 * 16:] != 0).sum()) == 0    # token 0 is zeros


# ---------------------------------------------------------------- readers

SPANS = [([(0, 1)], 0), ([(0, 16)], 0), ([(3, 40), (0, 0), (17, 1), (30, 63)], 5), ([(15, 33)] * 3, 0), ([(i % 40, 1) for i in range(50)], 2),
         ([(0, 0), (0, 300), (100, 7)], 1)]


def table_for(spans, bs, seed):
    g = gen(seed)
    need = [-(-(f + n) // bs) for f, n in spans]
    NB = sum(need) + 3
    perm = torch.randperm(NB, generator=g).to(torch.int32)
    tables = torch.full((len(spans), max(need + [1]) + 1), -7, dtype=torch.int32)      # unused entries: no block
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
    starts = torch.tensor([0] + [n for _, n in spans]).cumsum(0).to(torch.int32)
    first = torch.tensor([f for f, _ in spans], dtype=torch.int32)
    return tables, starts, first, NB


def places(spans, tables, bs):
    b, o = [], []
    for i, (f, n) in enumerate(spans):
        for p in range(f, f + n):
            b.append(int(tables[i, p // bs]))
            o.append(p % bs)
    return torch.tensor(b, dtype=torch.int64), torch.tensor(o, dtype=torch.int64)


def bf16_of(x, scale):
    """bf16(fp32(x * scale)) of exact float64 x (a code, or code * group scale)."""
    return (x.float() * scale).to(torch.bfloat16)


@pytest.mark.parametrize("spans,pad", SPANS)
@pytest.mark.parametrize("bs,Hk,form", [(16, 8, "native"), (32, 1, "shuffled"), (48, 3, "native"), (64, 2, "slots"),
                                        (128, 4, "shuffled"), (16, 2, "slots")])
def test_gather(spans, pad, bs, Hk, form):
    tables, starts, first, NB = table_for(spans, bs, 7)
    g = gen(8)
    kc = torch.randint(0, 256, (NB, Hk, 8, bs, 16), generator=g, dtype=torch.uint8)
    vc = torch.randint(0, 256, (NB, Hk, bs // 16, 128, 16) if form == "shuffled" else (NB, Hk, 128, bs), generator=g,
                       dtype=torch.uint8)
    b, o = places(spans, tables, bs)
    T = len(b) + pad
    n = torch.arange(len(b))
    k = kc[b, :, :, o].reshape(-1, Hk, 128).view(torch.float8_e4m3fn).double()
    v = vc[b, :, o // 16, :, o % 16] if form == "shuffled" else vc[b, :, :, o]
    v = v.contiguous().view(torch.float8_e4m3fn).double()
    k_out, v_out = (torch.full((T, Hk, 128), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    d = [x.to(DEV) for x in (tables, starts)]
    if form == "slots":
        ks, vs = (torch.rand(NB, Hk, bs, generator=g) for _ in range(2))
        pda.gather_cache_slot_scales(kc.to(DEV), vc.to(DEV), ks.to(DEV), vs.to(DEV), *d, T, first=first.to(DEV), k_out=k_out,
                                     v_out=v_out)
        fk, fv = ks[b, :, o][..., None], vs[b, :, o][..., None]
    else:
        pda.gather_cache(kc.to(DEV), vc.to(DEV), *d, T, 0.0371, 1.7, first=first.to(DEV), v_shuffled=form == "shuffled",
                         k_out=k_out, v_out=v_out)
        fk, fv = torch.tensor(0.0371), torch.tensor(1.7)
    for got, x, f in ((k_out, k, fk), (v_out, v, fv)):
        want = torch.cat([bf16_of(x, f), torch.full((pad, Hk, 128), 9.0, dtype=torch.bfloat16)])
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=-99.0), torch.nan_to_num(want, nan=-99.0))
    assert pda.query_device_status() == 0


@pytest.mark.parametrize("spans,pad", SPANS)
@pytest.mark.parametrize("bs,Hk", [(16, 8), (32, 1), (48, 3), (128, 2)])
def test_gather_fp4(spans, pad, bs, Hk):
    tables, starts, first, NB = table_for(spans, bs, 9)
    cache = U.random_cache4(NB, Hk, bs, 0.01, gen(10), wild=True)
    b, o = places(spans, tables, bs)
    T = len(b) + pad
    k_out, v_out = (torch.full((T, Hk, 128), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pda.gather_cache_fp4(cache.to(DEV), tables.to(DEV), starts.to(DEV), T, 0.0371, 1.7, first=first.to(DEV), k_out=k_out,
                         v_out=v_out)
    for got, kind, g in ((k_out, 0, 0.0371), (v_out, 1, 1.7)):
        want = bf16_of(U.read4(cache, bs, kind, b, o, 1.0)[0], torch.tensor(g))
        want = torch.cat([want, torch.full((pad, Hk, 128), 9.0, dtype=torch.bfloat16)])
        assert torch.equal(got.cpu(), want)
    assert pda.query_device_status() == 0


@pytest.mark.parametrize("form", ["e4m3", "fp4"])
def test_gather_bounds(form):
    """Rows outside the table row or the pool are zeros and are flagged; rows in front of the first sequence stay."""
    bs, Hk, NB = 16, 2, 4
    tables = torch.tensor([[1, 99], [-3, 2]], dtype=torch.int32, device=DEV)
    starts = torch.tensor([2, 36, 70], dtype=torch.int32, device=DEV)
    first = torch.tensor([-1, 10], dtype=torch.int32, device=DEV)
    T = 72
    outs = [torch.full((T, Hk, 128), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    if form == "fp4":
        cache = U.random_cache4(NB, Hk, bs, 0.01, gen(1)).to(DEV)
        pda.gather_cache_fp4(cache, tables, starts, T, 1.0, 1.0, first=first, k_out=outs[0], v_out=outs[1])
    else:
        kc, vc = (torch.full((NB, Hk, *s), 0x38, dtype=torch.uint8, device=DEV) for s in ((8, bs, 16), (128, bs)))
        pda.gather_cache(kc, vc, tables, starts, T, 1.0, 1.0, first=first, k_out=outs[0], v_out=outs[1])
    assert pda.query_device_status() == 64
    bad = torch.zeros(T, dtype=torch.bool)
    bad[2] = True                       # position -1
    bad[2 + 17:36] = True               # position 16 on: block 99, then past the row
    bad[36:36 + 6] = True               # positions 10 .. 15: block -3
    bad[36 + 22:70] = True              # position 32 on: past the row
    for out in outs:
        out = out.cpu()
        assert (out[:2] == 9).all() and (out[70:] == 9).all()
        assert (out[bad] == 0).all()
        good = ~bad
        good[:2] = good[70:] = False
        assert good.sum() == 16 + 16 and (out[good].abs().amax(-1) > 0).all() and (out[good] != 9).any()


def test_nothing_to_do():
    cache = torch.zeros(pda.fp4_cache_shape(2, 2, 16), dtype=torch.uint8, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    k, v = pda.gather_cache_fp4(cache, torch.zeros(0, 3, **i32), torch.zeros(1, **i32), 0, 1.0, 1.0)
    assert k.shape == (0, 2, 128)
    x = torch.zeros(0, 2, 128, dtype=torch.bfloat16, device=DEV)
    pda.reshape_and_cache_fp4(x, x, cache, torch.zeros(0, dtype=torch.int64, device=DEV), 1.0, 1.0)
    assert not cache.any()


def test_far_offsets():
    """Records, pages and scale rows past 2^32 bytes."""
    Hk, bs = 8, 16
    NB = (1 << 32) // (Hk * 128 * bs) + 500
    k, v = tokens(20, Hk, 5, "plain")
    slots = torch.cat([torch.arange(10) + (NB - 2) * bs + 3, torch.arange(10) + 40])
    tables = torch.tensor([[NB - 2, NB - 1], [2, 3]], dtype=torch.int32)
    starts, first = torch.tensor([0, 10, 20], dtype=torch.int32), torch.tensor([3, 8], dtype=torch.int32)
    d = [x.to(DEV) for x in (tables, starts)]
    cache = torch.empty(pda.fp4_cache_shape(NB, Hk, bs), dtype=torch.uint8, device=DEV)
    pda.reshape_and_cache_fp4(k, v, cache, slots.to(DEV), 0.01, 0.01)
    got = pda.gather_cache_fp4(cache, *d, 20, 0.01, 0.01, first=first.to(DEV))
    for x, y in zip((k, v), got):
        codes, scales = U.quantize_rows4(x.cpu(), 0.01)
        small = torch.zeros(pda.fp4_cache_shape(2, Hk, bs), dtype=torch.uint8)
        U.write4(small, bs, 0, torch.arange(20), codes, scales)
        n = torch.arange(20)
        want = bf16_of(U.read4(small, bs, 0, n // bs, n % bs, 1.0)[0], torch.tensor(0.01))
        assert torch.equal(torch.nan_to_num(y.cpu(), nan=-99.0), torch.nan_to_num(want, nan=-99.0))
    del cache
    kc = torch.empty(NB, Hk, 8, bs, 16, dtype=torch.uint8, device=DEV)
    vc = torch.empty(NB, Hk, 128, bs, dtype=torch.uint8, device=DEV)
    ks, vs = (torch.empty(NB, Hk, bs, device=DEV) for _ in range(2))
    pda.reshape_and_cache_slot_scales(k, v, kc, vc, ks, vs, slots.to(DEV))
    got = pda.gather_cache_slot_scales(kc, vc, ks, vs, *d, 20, first=first.to(DEV))
    for x, y in zip((k, v), got):
        codes, scales = U.quantize_rows8(x.cpu(), MIN)
        want = bf16_of(codes.view(torch.float8_e4m3fn).double(), scales[..., None])
        assert torch.equal(torch.nan_to_num(y.cpu(), nan=-99.0), torch.nan_to_num(want, nan=-99.0))
    assert pda.query_device_status() == 0


def test_captured_and_replayed():
    """A step of write and read back in a graph, replayed on other tokens at other slots, beside another stream."""
    bs, Hk, T = 16, 4, 33
    cache = torch.zeros(pda.fp4_cache_shape(20, Hk, bs), dtype=torch.uint8, device=DEV)
    k, v = (torch.zeros(T, Hk, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots = torch.zeros(T, dtype=torch.int64, device=DEV)
    tables, first = torch.zeros(T, 1, dtype=torch.int32, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
    starts = torch.arange(T + 1, dtype=torch.int32, device=DEV)
    k_out, v_out = (torch.zeros(T, Hk, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pda.reshape_and_cache_fp4(k, v, cache, slots, 0.01, 0.02)
        pda.gather_cache_fp4(cache, tables, starts, T, 0.01, 0.02, first=first, k_out=k_out, v_out=v_out)
    for seed in range(3):
        kk, vv = tokens(T, Hk, seed, "plain")
        s = torch.randperm(20 * bs, generator=gen(seed))[:T]
        k.copy_(kk)
        v.copy_(vv)
        slots.copy_(s)
        tables.copy_((s // bs)[:, None])
        first.copy_(s % bs)
        graph.replay()
        torch.cuda.synchronize()
        for x, y, g in ((kk, k_out, 0.01), (vv, v_out, 0.02)):
            codes, scales = U.quantize_rows4(x.cpu(), g)
            small = torch.zeros(pda.fp4_cache_shape(3, Hk, bs), dtype=torch.uint8)
            n = torch.arange(T)
            U.write4(small, bs, 0, n, codes, scales)
            want = bf16_of(U.read4(small, bs, 0, n // bs, n % bs, 1.0)[0], torch.tensor(g))
            assert torch.equal(torch.nan_to_num(y.cpu(), nan=-99.0), torch.nan_to_num(want, nan=-99.0))


def test_refusals_on_the_gpu():
    k, v = tokens(4, 2, 0, "plain")
    slots = torch.arange(4, device=DEV)
    cache = torch.zeros(pda.fp4_cache_shape(2, 2, 16), dtype=torch.uint8, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    tables, starts = torch.zeros(1, 2, **i32), torch.tensor([0, 4], **i32)
    bad_writes = [(k[:3], v, cache, slots), (k.float(), v, cache, slots), (k, v, cache[:, :1], slots), (k, v, cache.view(torch.int8), slots),
                  (k, v, cache, slots.int()), (k, v, cache[..., :100], slots), (k.transpose(1, 2), v.transpose(1, 2), cache, slots),
                  (k, v, cache, slots.cpu())]
    for a in bad_writes:
        with pytest.raises(pda.PdaError):
            pda.reshape_and_cache_fp4(*a, 0.1, 0.1)
    for a in [(cache, tables, starts[:1], 4), (cache, tables.long(), starts, 4), (cache, tables, starts, -1), (cache[0], tables, starts, 4)]:
        with pytest.raises(pda.PdaError):
            pda.gather_cache_fp4(*a, 0.1, 0.1)
    with pytest.raises(pda.PdaError):
        pda.gather_cache_fp4(cache, tables, starts, 4, 0.1, 0.1, k_out=torch.zeros(4, 2, 128, device=DEV))
    with pytest.raises(pda.PdaError):
        pda.gather_cache_fp4(cache, tables, starts, 4, 0.1, 0.1, first=torch.zeros(2, **i32))
    kc, vc = (torch.zeros(2, 2, *s, dtype=torch.uint8, device=DEV) for s in ((8, 16, 16), (128, 16)))
    ks = torch.zeros(2, 2, 16, device=DEV)
    for a in [(k, v, kc, vc, ks, ks[:1], slots), (k, v, kc, kc, ks, ks, slots), (k, v, kc, vc, ks.double(), ks, slots)]:
        with pytest.raises(pda.PdaError):
            pda.reshape_and_cache_slot_scales(*a)
    with pytest.raises(pda.PdaError) as e:
        pda.reshape_and_cache_slot_scales(k, v, kc, vc, ks, ks, slots, min_scale=0.0)
    assert e.value.status == pda.PDA_ERR_INVALID_ARG
    assert not cache.any() and not kc.any()


def test_writes_behind_a_decode():
    """A write right behind a decode that still reads the same slots: the decode sees what was there before. Batches whose tail
    kernel has nothing to join, beside one long sequence that keeps the decode busy."""
    S, H, Hk, bs, MB = 256, 8, 8, 16, 256
    g = gen(70)
    NB = MB + S
    tables = torch.arange(MB, dtype=torch.int32).repeat(S, 1)
    tables[1:, 0] = torch.arange(MB, NB - 1, dtype=torch.int32)
    lens = torch.full((S,), 5, dtype=torch.int32)
    lens[0] = MB * bs
    assert pda.plan_launches(S, H, Hk, MB, bs) >= 2
    kc = torch.randint(0, 0x70, (NB, Hk, 8, bs, 16), generator=g, dtype=torch.uint8)
    vc = torch.randint(0, 0x70, (NB, Hk, 128, bs), generator=g, dtype=torch.uint8)
    q = torch.randn(S, H, 128, generator=g).to(torch.bfloat16).to(DEV)
    tables, lens = tables.to(DEV), lens.to(DEV)
    T = MB * bs
    k, v = (torch.randn(T, Hk, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    slots = torch.arange(T, device=DEV)
    first = [t.to(DEV) for t in (kc, vc)]
    want = pda.decode(q, *first, tables, lens, 0.01, 0.01, 0.01)
    torch.cuda.synchronize()
    for i in range(20):
        caches = [t.clone() for t in first]
        scales = [torch.ones(NB, Hk, bs, device=DEV) for _ in range(2)]
        out = torch.empty_like(want)
        torch.cuda.synchronize()
        pda.decode(q, *caches, tables, lens, 0.01, 0.01, 0.01, out=out)
        pda.reshape_and_cache_slot_scales(k, v, *caches, *scales, slots)
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
    assert pda.query_device_status() == 0


@pytest.mark.parametrize("captured", [False, True])
def test_inputs_of_another_stream(captured):
    """Tokens that another stream makes, late, and an event tells of: written, read back and attended to in this one."""
    T, Hk, H, bs = 64, 2, 8, 16
    g = gen(80)
    src = [torch.randn(T, Hk, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    k, v = (torch.zeros_like(t) for t in src)
    busy = torch.randn(2048, 2048, device=DEV)
    work = torch.empty_like(busy)
    cache = torch.zeros(pda.fp4_cache_shape(4, Hk, bs), dtype=torch.uint8, device=DEV)
    tables = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    starts, lens = torch.tensor([0, T], dtype=torch.int32, device=DEV), torch.tensor([T], dtype=torch.int32, device=DEV)
    slots = torch.arange(T, device=DEV)
    q = torch.randn(1, H, 128, generator=g).to(torch.bfloat16).to(DEV)
    kb, vb = (torch.zeros(T, Hk, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    out = torch.zeros_like(q)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        kb.zero_()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for _ in range(8):
                torch.mm(busy, busy, out=work)
            k.copy_(src[0])
            v.copy_(src[1])
        out.zero_()
        main.wait_stream(side)
        pda.reshape_and_cache_fp4(k, v, cache, slots, 0.0043, 0.0043)
        pda.gather_cache_fp4(cache, tables, starts, T, 0.0043, 0.0043, k_out=kb, v_out=vb)
        pda.decode_fp4(q, cache, tables, lens, 128 ** -0.5, 0.0043, 0.0043, out=out)

    with torch.cuda.stream(main):
        pda.reserve_fp4(main)
        step()
        main.synchronize()
        want = [t.clone() for t in (cache, kb, vb, out)]
        assert out.abs().sum() > 0
        graph = None
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=main):
                step()
        for _ in range(10):
            for t in (k, v, cache, kb, vb, out):
                t.zero_()
            graph.replay() if captured else step()
            main.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((cache, kb, vb, out), want))
    codes, _ = U.quantize_rows4(src[0].cpu(), 0.0043)
    table, _, _ = U.Record(bs).tables()
    t = torch.arange(T)
    held = cache.cpu()[t // bs][:, :, :].gather(2, table[0][t % bs][:, None].expand(-1, Hk, -1)) >> (torch.arange(128) % 2 * 4) & 15
    assert torch.equal(held.to(torch.uint8), codes)
    assert pda.query_device_status() == 0


@pytest.mark.parametrize("T,Hk,bs,kind,layout", [(130, 37, 16, "run", "plain"), (70, 66, 32, "scattered", "heads_first"),
                                                 (4200, 1, 16, "blocks", "odd"), (33, 130, 128, "run", "packed")])
def test_write_heads_that_do_not_fill_a_block(T, Hk, bs, kind, layout):
    """The tiled writer where its last warps have no head."""
    test_write_slot_scales(T, Hk, bs, kind, layout, MIN)
