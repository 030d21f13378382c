"""The caches in fewer bits, on the CPU: refusals before any launch, and the plain forms the GPU tests rest on."""

import ctypes

import numpy as np
import pytest
import torch

import paged_kv_decode_pda_gb300 as pda
from paged_kv_decode_pda_gb300 import _binding as B
from paged_kv_decode_pda_gb300 import build
from tests import lowbits_util as U

A = 1 << 20          # a 16-byte aligned address nothing reads: every call below is refused on the host
INVALID, UNSUPPORTED, OK = pda.PDA_ERR_INVALID_ARG, pda.PDA_ERR_UNSUPPORTED, pda.PDA_OK
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pda.load()


def rows(base=A, tok=1024, head=128):
    return B._TokenRows(base, tok, head)


def write8(lib, k=rows(), v=rows(), kc=A, vc=A, ks=A, vs=A, slots=A, T=4, K=8, D=128, bs=16, NB=4, least=1e-6):
    return lib.pda_reshape_and_cache_slot_scales(ctypes.addressof(k) if k else None, ctypes.addressof(v) if v else None,
                                                 kc, vc, ks, vs, slots, T, K, D, bs, NB, least, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=rows(base=None)), INVALID), (dict(v=rows(base=A + 1)), INVALID),
    (dict(kc=None), INVALID), (dict(vc=A + 8), INVALID), (dict(ks=None), INVALID), (dict(vs=A + 2), INVALID),
    (dict(slots=None), INVALID), (dict(slots=A + 4), INVALID), (dict(T=-1), INVALID), (dict(K=0), INVALID),
    (dict(K=65536), UNSUPPORTED), (dict(D=64), UNSUPPORTED), (dict(D=0), INVALID), (dict(bs=24), UNSUPPORTED),
    (dict(bs=144), UNSUPPORTED), (dict(bs=0), INVALID), (dict(NB=-1), INVALID), (dict(NB=1 << 31), UNSUPPORTED),
    (dict(least=0.0), INVALID), (dict(least=-1.0), INVALID), (dict(least=NAN), INVALID), (dict(least=INF), INVALID),
    (dict(least=1e-38), UNSUPPORTED), (dict(T=0, k=rows(base=None), slots=None, kc=None), OK),
])
def test_write_slot_scales_refuses(lib, kw, status):
    assert write8(lib, **kw) == status


def write4(lib, k=rows(), v=rows(), c=A, slots=A, T=4, K=8, D=128, bs=16, NB=4, ks=0.01, vs=0.01):
    return lib.pda_reshape_and_cache_fp4(ctypes.addressof(k) if k else None, ctypes.addressof(v) if v else None, c, slots, T,
                                         K, D, bs, NB, ks, vs, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=rows(base=None)), INVALID), (dict(k=rows(base=A + 1)), INVALID), (dict(c=None), INVALID),
    (dict(c=A + 8), INVALID), (dict(slots=None), INVALID), (dict(slots=A + 4), INVALID), (dict(T=-1), INVALID),
    (dict(D=256), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(NB=-1), INVALID), (dict(ks=0.0), INVALID),
    (dict(vs=-0.1), INVALID), (dict(ks=NAN), INVALID), (dict(vs=INF), INVALID), (dict(ks=2.0 ** -101), UNSUPPORTED),
    (dict(vs=2.0 ** 101), UNSUPPORTED), (dict(T=0, c=None), OK),
])
def test_write_fp4_refuses(lib, kw, status):
    assert write4(lib, **kw) == status


def gather(lib, kind, ko=A, vo=A + 4096, kc=A, vc=A, ksc=A, vsc=A, tab=A, st=A, fi=A, T=4, S=2, K=8, D=128, bs=16, MB=4, NB=4, ks=0.1,
           vs=0.1, layout=0):
    tail = (tab, st, fi, T, S, K, D, bs, MB, NB)
    if kind == "e4m3":
        return lib.pda_gather_cache(ko, vo, kc, vc, *tail, ks, vs, layout, None)
    if kind == "slots":
        return lib.pda_gather_cache_slot_scales(ko, vo, kc, vc, ksc, vsc, *tail, None)
    return lib.pda_gather_cache_fp4(ko, vo, kc, *tail, ks, vs, None)


@pytest.mark.parametrize("kind", ["e4m3", "slots", "fp4"])
@pytest.mark.parametrize("kw,status", [
    (dict(ko=None), INVALID), (dict(vo=A + 8), INVALID), (dict(vo=A), INVALID), (dict(kc=None), INVALID), (dict(kc=A + 4), INVALID),
    (dict(tab=None), INVALID), (dict(tab=A + 2), INVALID), (dict(st=None), INVALID), (dict(st=A + 1), INVALID),
    (dict(fi=A + 2), INVALID), (dict(T=-1), INVALID), (dict(S=-1), INVALID), (dict(K=0), INVALID), (dict(K=65536), UNSUPPORTED),
    (dict(D=64), UNSUPPORTED), (dict(bs=20), UNSUPPORTED), (dict(MB=-1), INVALID), (dict(MB=1 << 27), UNSUPPORTED),
    (dict(NB=-1), INVALID), (dict(NB=1 << 31), UNSUPPORTED), (dict(T=0, ko=None, st=None), OK), (dict(S=0, ko=None, st=None), OK),
])
def test_gather_refuses(lib, kind, kw, status):
    assert gather(lib, kind, **kw) == status


@pytest.mark.parametrize("kind,kw,status", [
    ("e4m3", dict(vc=None), INVALID), ("e4m3", dict(layout=2), INVALID), ("e4m3", dict(ks=NAN), INVALID),
    ("e4m3", dict(vs=INF), INVALID), ("slots", dict(vc=A + 8), INVALID), ("slots", dict(ksc=None), INVALID),
    ("slots", dict(vsc=A + 2), INVALID), ("fp4", dict(ks=INF), INVALID), ("fp4", dict(vs=NAN), INVALID),
])
def test_gather_refuses_by_kind(lib, kind, kw, status):
    assert gather(lib, kind, **kw) == status


def decode(lib, out=A, q=A, c=A, tab=A, lens=A, S=2, H=32, K=8, D=128, bs=16, MB=4, NB=4, scale=0.1, ks=0.1, vs=0.1, window=0,
           sinks=None, dt=0, os=1.0):
    return lib.pda_decode_fp4(out, q, c, tab, lens, S, H, K, D, bs, MB, NB, scale, ks, vs, window, sinks, dt, os, None)


@pytest.mark.parametrize("kw,status", [
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(c=None), INVALID), (dict(tab=None), INVALID),
    (dict(lens=None), INVALID), (dict(out=A + 8), INVALID), (dict(q=A + 2), INVALID), (dict(c=A + 4), INVALID),
    (dict(tab=A + 2), INVALID), (dict(lens=A + 1), INVALID), (dict(sinks=A + 2), INVALID), (dict(S=-1), INVALID),
    (dict(H=33), INVALID), (dict(H=72), UNSUPPORTED), (dict(D=64), UNSUPPORTED), (dict(bs=24), UNSUPPORTED),
    (dict(bs=256), UNSUPPORTED), (dict(S=65536), UNSUPPORTED), (dict(MB=1 << 27), UNSUPPORTED), (dict(NB=0), INVALID),
    (dict(NB=-1), INVALID), (dict(NB=1 << 31), UNSUPPORTED), (dict(S=65535, MB=40000), UNSUPPORTED), (dict(window=-1), INVALID),
    (dict(dt=2), INVALID), (dict(dt=1, os=0.0), INVALID), (dict(dt=1, os=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(ks=NAN), INVALID), (dict(vs=INF), INVALID), (dict(S=0, q=None, c=None, NB=0), OK),
])
def test_decode_fp4_refuses(lib, kw, status):
    assert decode(lib, **kw) == status


def test_binding_refuses_cpu_tensors(lib):
    key = torch.zeros(2, 1, 128, dtype=torch.bfloat16)
    cache = torch.zeros(pda.fp4_cache_shape(3, 1, 16), dtype=torch.uint8)
    tables, starts = torch.zeros(1, 2, dtype=torch.int32), torch.tensor([0, 2], dtype=torch.int32)
    slots = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(pda.PdaError):
        pda.reshape_and_cache_fp4(key, key, cache, slots, 0.1, 0.1)
    with pytest.raises(pda.PdaError):
        pda.gather_cache_fp4(cache, tables, starts, 2, 0.1, 0.1)
    with pytest.raises(pda.PdaError):
        pda.decode_fp4(key, cache, tables, starts[:1], 0.1, 0.1, 0.1)


# ------------------------------------------------------------ plain forms

def test_codes_are_the_nearest():
    """Every bf16 magnitude near the grid against each value of the grid, by distance in exact arithmetic."""
    from fractions import Fraction
    for grid in (U.E2M1, U.E4M3):
        unit = float(np.float32(0.0137))
        for x in np.concatenate([grid * unit, (grid[1:] + grid[:-1]) / 2 * unit, grid * unit * 1.01, [0.0, grid[-1] * unit * 5]]):
            code = int(U.nearest_code(np.array([x]), np.array([unit]), grid)[0])
            ratio = min(Fraction(x) / Fraction(unit), Fraction(float(grid[-1])))
            far = [abs(ratio - Fraction(float(v))) for v in grid]
            assert far[code] == min(far)
            assert far.count(min(far)) == 1 or code % 2 == 0


def test_record_places_are_a_permutation():
    for bs in (16, 48, 128):
        c, shift, s = U.Record(bs).tables()
        nibbles = sorted((2 * c + (shift // 4)).flatten().tolist())
        assert nibbles == list(range(2 * 128 * bs))
        assert sorted(s.flatten().tolist()) == list(range(128 * bs, 144 * bs))


def test_values_come_back():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(40, 2, 128, generator=g).to(torch.bfloat16)
    cache = torch.zeros(pda.fp4_cache_shape(3, 2, 16), dtype=torch.uint8)
    slots = torch.randperm(48, generator=g)[:40]
    codes, scales = U.quantize_rows4(x, 0.001)
    U.write4(cache, 16, 1, slots, codes, scales)
    y = U.read4(cache, 16, 1, slots // 16, slots % 16, 0.001)[1]
    # half an e2m1 step is at most 1 of 6 of the group's largest (4 .. 6), and its scale moves by 2^-4
    amax = x.double().abs().view(40, 2, 8, 16).amax(-1, keepdim=True).expand(-1, -1, -1, 16).reshape(40, 2, 128)
    # nothing lies past 448 * 6 * g: a group scale saturates at 448 and a code at 6, so what is larger becomes that value
    top = 448 * 6 * float(np.float32(0.001))
    assert ((y - x.double().clamp(-top, top)).abs() <= amax * (1 / 6 + 2.0 ** -4)).all()
