"""The operators around the decode call, on the CPU: refusals before any launch, and the rotary frequencies."""

import ctypes
import math

import pytest
import torch

import paged_kv_decode_pda_gb300 as pda
from paged_kv_decode_pda_gb300 import _binding as B
from paged_kv_decode_pda_gb300 import build

A = 1 << 20          # a 16-byte aligned address nothing reads: every call below is refused on the host
INVALID, UNSUPPORTED = pda.PDA_ERR_INVALID_ARG, pda.PDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pda.load()


def heads(src=A, dst=A, tok=1024, head=128, n=8):
    return B._RopeHeads(src, dst, tok, head, tok, head, n)


def freqs(n=64, value=0.5):
    return (ctypes.c_double * max(n, 1))(*([value] * n))


def rope_call(lib, q=None, k=heads(), pos=A, T=4, D=128, f=freqs(), rot=128, mag=1.0):
    q = heads() if q is None else q
    return lib.pda_rope(ctypes.addressof(q) if q else None, ctypes.addressof(k) if k else None, pos, T, D,
                        ctypes.addressof(f) if f else None, rot, 0, mag, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=heads(src=None)), INVALID), (dict(q=heads(dst=None)), INVALID), (dict(k=heads(src=None)), INVALID),
    (dict(k=heads(dst=None)), INVALID), (dict(q=heads(n=0)), INVALID), (dict(k=heads(n=-1)), INVALID),
    (dict(q=heads(n=70000)), UNSUPPORTED), (dict(q=heads(src=A + 1)), INVALID), (dict(pos=None), INVALID),
    (dict(pos=A + 4), INVALID), (dict(T=-1), INVALID), (dict(D=64), UNSUPPORTED), (dict(D=0), INVALID),
    (dict(f=None), INVALID), (dict(rot=127), INVALID), (dict(rot=-2), INVALID), (dict(rot=130), UNSUPPORTED),
    (dict(mag=float("nan")), INVALID), (dict(f=freqs(value=float("nan"))), INVALID),
    (dict(f=freqs(value=3.2)), INVALID), (dict(f=freqs(value=float("inf"))), INVALID),
])
def test_rope_refuses(lib, kw, status):
    assert rope_call(lib, **kw) == status


def test_rope_without_tokens_is_a_noop(lib):
    assert rope_call(lib, T=0, q=heads(src=None, dst=None), pos=None) == pda.PDA_OK


def cache_call(lib, q=heads(), k=heads(), v=heads(), pos=A, slots=A, T=4, D=128, rot=128, kc=A, vc=A, bs=16, NB=4,
               ks=0.1, vs=0.1, layout=0):
    f = freqs()
    return lib.pda_rope_and_cache(ctypes.addressof(q), ctypes.addressof(k) if k else None,
                                  ctypes.addressof(v) if v else None, pos, slots, T, D, ctypes.addressof(f), rot, 0,
                                  1.0, kc, vc, bs, NB, ks, vs, layout, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(v=heads(n=4)), INVALID), (dict(k=heads(n=0)), INVALID),
    (dict(v=heads(src=None)), INVALID), (dict(slots=None), INVALID), (dict(slots=A + 4), INVALID),
    (dict(kc=None), INVALID), (dict(vc=A + 8), INVALID), (dict(bs=0), INVALID), (dict(bs=24), UNSUPPORTED),
    (dict(bs=144), UNSUPPORTED), (dict(NB=-1), INVALID), (dict(ks=0.0), INVALID), (dict(vs=float("inf")), INVALID),
    (dict(layout=2), INVALID), (dict(D=256), UNSUPPORTED), (dict(rot=132), UNSUPPORTED),
])
def test_rope_and_cache_refuses(lib, kw, status):
    assert cache_call(lib, **kw) == status


def extend_call(lib, out=A, q=A, k=A, v=A, tables=A, lens=A, starts=A, T=4, S=2, H=8, Hk=2, D=128, bs=16, MB=4,
                scale=0.1, ks=0.05, vs=0.05, window=0, layout=0, sinks=None, dtype=0, oscale=1.0):
    return lib.pda_extend(out, q, k, v, tables, lens, starts, T, S, H, Hk, D, bs, MB, scale, ks, vs, window, layout,
                          sinks, dtype, oscale, None)


@pytest.mark.parametrize("kw,status", [
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(tables=None), INVALID), (dict(lens=None), INVALID), (dict(starts=None), INVALID), (dict(q=A + 8), INVALID),
    (dict(starts=A + 2), INVALID), (dict(T=-1), INVALID), (dict(S=-1), INVALID), (dict(S=70000), UNSUPPORTED),
    (dict(H=18), UNSUPPORTED), (dict(H=7), INVALID), (dict(D=64), UNSUPPORTED), (dict(bs=24), UNSUPPORTED),
    (dict(bs=256), UNSUPPORTED), (dict(MB=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(ks=float("inf")), INVALID), (dict(window=-1), INVALID), (dict(layout=3), INVALID), (dict(dtype=2), INVALID),
    (dict(dtype=1, oscale=0.0), INVALID), (dict(dtype=1, oscale=float("nan")), INVALID), (dict(sinks=A + 2), INVALID),
    (dict(T=1 << 30, H=16), UNSUPPORTED),
])
def test_extend_refuses(lib, kw, status):
    assert extend_call(lib, **kw) == status


def test_reserve_extend_refuses(lib):
    assert lib.pda_reserve_extend(-1, 1, 8, 2, 4, 16, None) == INVALID
    assert lib.pda_reserve_extend(4, 1, 7, 2, 4, 16, None) == INVALID
    assert lib.pda_reserve_extend(4, 1, 8, 2, 4, 24, None) == UNSUPPORTED
    assert lib.pda_reserve_extend(1 << 30, 1, 16, 2, 4, 16, None) == UNSUPPORTED
    assert lib.pda_reserve_extend(0, 0, 8, 2, 4, 16, None) == pda.PDA_OK


def test_extend_of_nothing_is_a_noop(lib):
    assert extend_call(lib, T=0, out=None, q=None) == pda.PDA_OK
    assert extend_call(lib, S=0, tables=None, lens=None, starts=None) == pda.PDA_OK


def table(**kw):
    d = dict(ref_counts=A, block_tables=A, seq_lens=A, num_blocks=8, num_rows=4, max_blocks=4, block_size=16)
    d.update(kw)
    return B._PageTable(*[d[f] for f, _ in B._PageTable._fields_])


BAD_TABLES = [
    (dict(ref_counts=None), INVALID), (dict(block_tables=None), INVALID), (dict(seq_lens=None), INVALID),
    (dict(ref_counts=A + 2), INVALID), (dict(num_blocks=-1), INVALID), (dict(num_rows=-1), INVALID),
    (dict(max_blocks=-1), INVALID), (dict(block_size=0), INVALID), (dict(block_size=24), UNSUPPORTED),
    (dict(block_size=144), UNSUPPORTED), (dict(max_blocks=1 << 30), UNSUPPORTED),
    (dict(num_blocks=1 << 31), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD_TABLES)
def test_page_calls_refuse_tables(lib, kw, status):
    t = table(**kw)
    p = ctypes.addressof(t)
    assert lib.pda_grow_pages(p, A, A, 1, None) == status
    assert lib.pda_fork_pages(p, A, A, 1, None, 0, None) == status
    assert lib.pda_free_pages(p, A, 1, None) == status
    assert lib.pda_compact_pages(p, None, 0, None, None) == status


def test_page_calls_refuse_arguments(lib):
    t = table()
    p = ctypes.addressof(t)
    assert lib.pda_grow_pages(None, A, A, 1, None) == INVALID
    assert lib.pda_grow_pages(p, None, A, 1, None) == INVALID
    assert lib.pda_grow_pages(p, A, A + 1, 1, None) == INVALID
    assert lib.pda_grow_pages(p, A, A, -1, None) == INVALID
    assert lib.pda_fork_pages(p, A, None, 1, None, 0, None) == INVALID
    assert lib.pda_fork_pages(p, A, A, 1, None, 1, None) == INVALID
    assert lib.pda_free_pages(p, None, 1, None) == INVALID
    assert lib.pda_compact_pages(p, None, 0, A + 2, None) == INVALID
    assert lib.pda_reserve_pages(-1, 1, 1, None) == INVALID
    assert lib.pda_reserve_pages(1 << 31, 1, 1, None) == UNSUPPORTED
    for base, size in ((None, 64), (A + 8, 64), (A, 24), (A, 0)):
        arr = (B._PageArray * 1)(B._PageArray(base, size))
        for st in (lib.pda_copy_pages(ctypes.addressof(arr), 1, A, A, 1, 8, None),
                   lib.pda_fork_pages(p, A, A, 1, ctypes.addressof(arr), 1, None),
                   lib.pda_compact_pages(p, ctypes.addressof(arr), 1, None, None)):
            assert st == INVALID
    arr = (B._PageArray * 1)(B._PageArray(A, 64))
    assert lib.pda_copy_pages(ctypes.addressof(arr), 1, None, A, 1, 8, None) == INVALID
    assert lib.pda_copy_pages(ctypes.addressof(arr), -1, A, A, 1, 8, None) == INVALID
    assert lib.pda_copy_pages(ctypes.addressof(arr), 1, A, A, -1, 8, None) == INVALID
    # nothing to do: no pointer is looked at
    assert lib.pda_grow_pages(p, None, None, 0, None) == pda.PDA_OK
    assert lib.pda_fork_pages(p, None, None, 0, None, 0, None) == pda.PDA_OK
    assert lib.pda_free_pages(p, None, 0, None) == pda.PDA_OK
    assert lib.pda_copy_pages(None, 0, None, None, 5, 8, None) == pda.PDA_OK


def test_binding_refuses_types_and_shapes(lib):
    bf, f64 = torch.bfloat16, torch.float64
    q, pos, f = torch.zeros(3, 4, 128, dtype=bf), torch.zeros(3, dtype=torch.int64), torch.ones(64, dtype=f64)
    for args in ((q.float(), None, pos, f), (q, q[:2], pos, f), (q, None, pos.int(), f), (q, None, pos[:2], f),
                 (q, None, pos, f.float()), (q.transpose(1, 2), None, pos, f)):
        with pytest.raises(pda.PdaError):
            pda.rope(*args)
    i32 = torch.int32
    refs, tab, lens = torch.zeros(8, dtype=i32), torch.zeros(4, 3, dtype=i32), torch.zeros(4, dtype=i32)
    rows = torch.zeros(2, dtype=i32)
    for args in ((refs, tab, lens[:3], rows, rows), (refs.long(), tab, lens, rows, rows),
                 (refs, tab.T, lens, rows, rows), (refs, tab, lens, rows, rows[:1]),
                 (refs, tab, lens, rows.long(), rows)):
        with pytest.raises(pda.PdaError):
            pda.grow_pages(*args, 16)
    with pytest.raises(pda.PdaError):
        pda.rope_frequencies(127)
    with pytest.raises(pda.PdaError):
        pda.rope_frequencies(0)


# ------------------------------------------------------------- frequencies

def test_plain_frequencies(lib):
    f, mag = pda.rope_frequencies(64, 10000.0)
    assert mag == 1.0 and f.dtype == torch.float64
    assert f.tolist() == pytest.approx([10000.0 ** (-i / 32) for i in range(32)], rel=1e-15)


def test_linear_and_base_frequencies(lib):
    plain, _ = pda.rope_frequencies(128)
    lin, _ = pda.rope_frequencies(128, scaling=pda.PDA_ROPE_LINEAR, factor=8)
    assert (lin * 8 - plain).abs().max() < 1e-15
    base, _ = pda.rope_frequencies(128, scaling=pda.PDA_ROPE_BASE, factor=8)
    assert base[0] == plain[0] and base[-1].item() == pytest.approx(plain[-1].item() / 8, rel=1e-12)


def test_ramp_frequencies(lib):
    L, s = 4096.0, 16.0
    plain, _ = pda.rope_frequencies(128)
    f, mag = pda.rope_frequencies(128, scaling=pda.PDA_ROPE_RAMP, factor=s, original_length=L)
    assert mag == pytest.approx(0.1 * math.log(s) + 1)
    turns = L * plain / (2 * math.pi)
    ratio = f / plain
    assert (ratio[turns > 40] == 1).all() and ((ratio[turns < 0.8] * s - 1).abs() < 1e-12).all()
    assert (ratio[1:] <= ratio[:-1] + 1e-15).all()


def test_band_frequencies(lib):
    L, s = 8192.0, 8.0
    plain, _ = pda.rope_frequencies(128, 500000.0)
    f, mag = pda.rope_frequencies(128, 500000.0, scaling=pda.PDA_ROPE_BANDS, factor=s, original_length=L)
    assert mag == 1.0
    for a, b in zip(plain.tolist(), f.tolist()):
        wave = 2 * math.pi / a
        if wave < L / 4:
            want = a
        elif wave > L:
            want = a / s
        else:
            t = (L / wave - 1) / 3
            want = (1 - t) * a / s + t * a
        assert b == pytest.approx(want, rel=1e-12)


@pytest.mark.parametrize("kw", [dict(rot_dim=128, base=1.0), dict(rot_dim=128, base=float("nan")),
                                dict(rot_dim=130), dict(rot_dim=128, scaling=5), dict(rot_dim=128, scaling=1, factor=0.5),
                                dict(rot_dim=128, scaling=3, factor=2.0), dict(rot_dim=2, scaling=2, factor=2.0),
                                dict(rot_dim=128, scaling=4, factor=2.0, original_length=64, low=4.0, high=4.0)])
def test_frequencies_refuse(lib, kw):
    with pytest.raises(pda.PdaError):
        pda.rope_frequencies(**kw)


# ----------------------------------------------- the tests' own references

def test_the_references_agree_with_worked_cases():
    from tests import ops_util as O
    x = torch.zeros(1, 1, 128)
    x[0, 0, 0], x[0, 0, 2] = 1.0, 5.0
    y = O.rope64(x, torch.tensor([1]), torch.tensor([math.pi / 2, 0.0], dtype=torch.float64), 2.0)
    assert abs(y[0, 0, 0] + 10) < 1e-14 and abs(y[0, 0, 2] - 2) < 1e-14     # pair (0, 2): (1, 5) -> (-5, 1) * 2
    y = O.rope64(x, torch.tensor([1]), torch.tensor([math.pi / 2], dtype=torch.float64), 1.0, True)
    assert abs(y[0, 0, 1] - 1) < 1e-15 and y[0, 0, 2] == 5
    # one token sees itself alone; a row in front of the cache sees nothing
    c = O.Chunk([(2, 1), (1, 1)], 2, 1)
    out, _ = c.exact()
    _, v = c.keys_values(1)
    assert (out[0] == 0).all() and (out[2] - v[0]).abs().max() < 1e-12
    p = O.Pool(4, 3, 4, 16)
    p.grow([0], [20])
    p.fork([0], [1])
    assert p.tables[1][:2] == [0, 2] and p.refs == [2, 1, 1, 0] and p.moves == [(1, 2)]
    p.free([0, 0])
    assert p.refs == [1, 0, 1, 0]
    p.compact()
    assert p.refs == [1, 1, 0, 0] and p.tables[1][:2] == [0, 1] and p.moves == [(2, 1)]


@pytest.mark.parametrize("rot,base,L,factor,low,high", [
    (128, 10000.0, 4096.0, 16.0, 1.0, 32.0), (64, 500000.0, 8192.0, 8.0, 1.0, 32.0), (96, 10000.0, 2048.0, 4.0, 2.0, 20.0),
    (32, 100.0, 4096.0, 4.0, 1.0, 32.0)])
def test_ramp_between_the_bands(lib, rot, base, L, factor, low, high):
    # over whole pair indices: from the last that makes `high` turns or more to the first that makes `low` or fewer
    # (the indices go on past the last pair)
    f, _ = pda.rope_frequencies(rot, base, scaling=pda.PDA_ROPE_RAMP, factor=factor, original_length=L, low=low, high=high)
    turns = [L * base ** (-2 * i / rot) / (2 * math.pi) for i in range(rot)]
    first = max([i for i in range(rot) if turns[i] >= high], default=0)
    last = min([i for i in range(rot) if turns[i] <= low], default=rot - 1)
    assert first < last
    for i, got in enumerate(f.tolist()):
        t = min(1.0, max(0.0, (i - first) / (last - first)))
        plain = base ** (-2 * i / rot)
        assert got == pytest.approx(plain * (1 - t) + plain / factor * t, rel=1e-12), i
