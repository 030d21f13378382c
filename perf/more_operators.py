"""Cases of the operators that keep a paged cache in fewer bits: the writers that find the scales of what they write, the
readers that give its values back, and the decode attention over a cache of 4 bits a value.

``run`` makes one pass: in plain torch operations where ``own`` is false, through the package's calls where it is true.

A 4-bit cache is uint8 ``[blocks, kv_heads, 144 * block_size]``. The record of a block and kv head holds, one after the
other: K codes ``[block_size][64]`` (byte j: dims 2j low, 2j+1 high, e2m1), V codes likewise with the two 32-byte halves
of a token exchanged where bit 1 of its slot is set, K scales ``[block_size][8]`` (e4m3, one per 16 dims), and V scales
``[block_size / 16][8][16]`` whose last index is 4 * ((t & 3) ^ (t >> 2 & 1)) + (t >> 2) for slot t of 16. A value is
e2m1 * block scale * tensor scale.
"""

from __future__ import annotations

import math
import random

import torch

own = False

D = 128
FP8 = torch.float8_e4m3fn
DEV = "cuda"
MIN_SCALE = 2.0 ** -20
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step's new tokens, each row with its own scale: a padded batch of 256 at scattered slots
        dict(name="write8-step-256", op="write8", tokens=256, kv_heads=8, block=16, pad=19, runs=False, packed=False),
        # a prefill of whole blocks, keys and values out of the packed projection
        dict(name="write8-prefill-8192", op="write8", tokens=8192, kv_heads=8, block=64, pad=0, runs=True, packed=True),
        # a finished sequence handed on: one table, one scale for the tensor
        dict(name="read8-one-1000", op="read8", seqs=1, ctx=1000, ctx_lo=1000, kv_heads=8, block=16, skip=0, slot=False,
             shuffled=False, pad=0, shape=1),
        # contexts of a batch of continuations, per-row scales, the shared beginnings left out
        dict(name="read8-slots-32", op="read8", seqs=32, ctx=4000, ctx_lo=1, kv_heads=8, block=16, skip=512, slot=True,
             shuffled=False, pad=7, shape=2),
        # a small step's tokens into 4 bits, and their values for the step's own attention
        dict(name="store4-step-16", op="store4", tokens=16, kv_heads=8, block=16, runs=False, packed=False),
        # a long prompt, stored and read back in the values that later steps will see
        dict(name="store4-prefill-16384", op="store4", tokens=16384, kv_heads=8, block=16, runs=True, packed=True),
        # a short context out of 4 bits
        dict(name="read4-one-512", op="read4", seqs=1, ctx=512, ctx_lo=512, kv_heads=8, block=16, skip=0, pad=0, shape=3),
        # ragged contexts of a batch
        dict(name="read4-ragged-64", op="read4", seqs=64, ctx=4000, ctx_lo=1, kv_heads=8, block=64, skip=100, pad=3,
             shape=4),
        # the smallest serving batch; latency
        dict(name="decode4-16x1024", op="decode4", seqs=16, ctx=1024, ctx_lo=1024, heads=32, kv_heads=8, block=16,
             window=0, sinks=False, shape=5),
        # the large batch at one length
        dict(name="decode4-256x4096", op="decode4", seqs=256, ctx=4096, ctx_lo=4096, heads=32, kv_heads=8, block=16,
             window=0, sinks=False, shape=6),
        # the large batch, ragged
        dict(name="decode4-256x1to4000", op="decode4", seqs=256, ctx=4000, ctx_lo=1, heads=40, kv_heads=8, block=16,
             window=0, sinks=False, shape=7),
        # two long contexts, large blocks, sinks, wide groups
        dict(name="decode4-2x131072", op="decode4", seqs=2, ctx=131072, ctx_lo=131072, heads=64, kv_heads=8, block=64,
             window=0, sinks=True, shape=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("write8", "read8", "store4", "read4", "decode4", "decode4"))
    kv = rng.choice((1, 2, 4, 8))
    block = rng.choice((16, 16, 32, 48, 64, 128))
    if op in ("write8", "store4"):
        runs = rng.random() < 0.5
        c = dict(op=op, tokens=_log(rng, 1, 8192), kv_heads=kv, block=block, runs=runs, packed=rng.random() < 0.5)
        if op == "write8":
            c["pad"] = 0 if runs else _log(rng, 1, 40) - 1
        return c
    if op in ("read8", "read4"):
        ctx = _log(rng, 1, 4000)
        c = dict(op=op, seqs=_log(rng, 1, 24), ctx=ctx, ctx_lo=ctx if rng.random() < 0.4 else 0, kv_heads=kv, block=block,
                 skip=rng.choice((0, _log(rng, 1, 600))), pad=rng.choice((0, 0, 5)), shape=rng.randrange(1 << 20))
        if op == "read8":
            c.update(slot=rng.random() < 0.5, shuffled=rng.random() < 0.3)
            if c["slot"]:
                c["shuffled"] = False
        return c
    ctx = _log(rng, 1, 65536)
    seqs = _log(rng, 1, max(1, min(256, 256 * 4096 // ctx)))
    return dict(op=op, seqs=seqs, ctx=ctx, ctx_lo=ctx if rng.random() < 0.4 else 0,
                heads=kv * rng.choice((1, 2, 3, 4, 5, 7, 8)), kv_heads=kv, block=block,
                window=rng.choice((0, 0, 1, _log(rng, 2, 4096))), sinks=rng.random() < 0.3, shape=rng.randrange(1 << 20))


def _lengths(case):
    rng = random.Random(case["shape"])
    return [rng.randint(case["ctx_lo"], case["ctx"]) for _ in range(case["seqs"])]


def _spans(case):
    """(first position, tokens) of each sequence that is read."""
    rng = random.Random(case["shape"] + 1)
    out = []
    for n in _lengths(case):
        first = min(n, rng.randint(0, case["skip"]))
        out.append((first, n - first))
    if not any(n for _, n in out):
        out[0] = (out[0][0], 1)
    return out


def work(case):
    op, K, B = case["op"], case["kv_heads"], case["block"]
    if op == "write8":
        w = case["tokens"] - min(case["pad"], case["tokens"] - 1)
        return {"bytes": w * K * (4 * D + 2 * D + 8) + 8 * case["tokens"], "flops": 4 * w * K * D}
    if op == "store4":
        T = case["tokens"]
        return {"bytes": T * K * (4 * D + 144 + 144 + 4 * D) + 8 * T, "flops": 8 * T * K * D}
    if op in ("read8", "read4"):
        row = 144 if op == "read4" else 2 * D + (8 if case["slot"] else 0)
        n = sum(m for _, m in _spans(case))
        pages = sum(-(-(f + m) // B) - f // B for f, m in _spans(case) if m)
        return {"bytes": n * K * (row + 4 * D) + 4 * pages + 8 * case["seqs"], "flops": 2 * n * K * D}
    seen = pages = 0
    for n in _lengths(case):
        lo = max(0, n - case["window"]) if case["window"] else 0
        seen += n - lo
        pages += -(-n // B) - lo // B
    return {"bytes": seen * K * 144 + case["seqs"] * (case["heads"] * D * 4 + 4) + 4 * pages,
            "flops": seen * case["heads"] * 4 * D}


# ------------------------------------------------------- formats, plainly

def _to_e4m3(x):
    """The e4m3 value next to each 64-bit x (ties to even, saturating, NaN kept), as the type."""
    y = x.abs().clamp(max=448.0)
    m, _ = torch.frexp(y)
    step = torch.where(y < 2.0 ** -6, 2.0 ** -9, y / m / 16)        # y / m is a power of two
    return ((y / step).round_() * step).copysign(x).to(FP8)


def _to_e2m1(x):
    """The e2m1 code next to each 64-bit x (ties to even, saturating)."""
    y = x.abs().clamp(max=6.0)
    code = torch.where(y < 2, (2 * y).round(), torch.where(y < 4, y.round() + 2, (y / 2).round() + 4))
    return code.to(torch.uint8) | (torch.signbit(x).to(torch.uint8) << 3)


def _over(x, y):
    """x / y for a number y. (A number would be multiplied by as its reciprocal, which moves ties.)"""
    return x / torch.full_like(x, y)


def _finite_amax(x):
    return torch.where(x.isfinite(), x.abs(), 0.0).amax(-1, keepdim=True)


def _quantize4(x, scale):
    """Rows [..., 128] -> (bytes [..., 64], block scales [..., 8] as e4m3)."""
    x = x.double().unflatten(-1, (8, 16))
    s = _to_e4m3(_over(_finite_amax(x), 6.0 * scale))
    unit = s.double() * scale
    code = _to_e2m1(torch.where(unit > 0, x / unit, 0.0).copysign(x)).flatten(-2)
    s = torch.where(x.isnan().any(-1, keepdim=True), math.nan, s.float()).to(FP8)
    return code[..., 0::2] | (code[..., 1::2] << 4), s[..., 0]


def _swap_halves(v, slot):
    """V bytes [..., 64] of slots: the halves change places where bit 1 of the slot is set (its own inverse)."""
    return torch.where((slot & 2).bool()[..., None], torch.cat([v[..., 32:], v[..., :32]], -1), v)


def _scale_place(t):
    return 4 * ((t & 3) ^ (t >> 2 & 1)) + (t >> 2)


def _sections(cache, block):
    """Views of a 4-bit cache: K codes, V codes [NB, K, bs, 64], K scales [NB, K, bs, 8], V scales [NB, K, bs/16, 8, 16]."""
    B = block
    kc, vc, ks, vs = cache.split([64 * B, 64 * B, 8 * B, 8 * B], -1)
    return (kc.unflatten(-1, (B, 64)), vc.unflatten(-1, (B, 64)), ks.unflatten(-1, (B, 8)),
            vs.unflatten(-1, (B // 16, 8, 16)))


def _values4(code, s, scale):
    """Bytes [..., 64] and e4m3 scale bytes [..., 8] -> values in 32 bits [..., 128]."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
    x = torch.stack([lut[(code & 15).int()], lut[(code >> 4).int()]], -1).flatten(-2).unflatten(-1, (8, 16))
    return (x * s.contiguous().view(FP8).float()[..., None]).flatten(-2) * scale


def _pages4(cache, ids, block, k_scale, v_scale):
    """Values of the pages ``ids`` [...]: K and V [..., K, bs, 128]."""
    kc, vc, ks, vs = _sections(cache[ids], block)
    t = torch.arange(block, device=DEV)
    vc = _swap_halves(vc, t)
    vs = vs[..., _scale_place(t[:16])].transpose(-1, -2).flatten(-3, -2)
    return _values4(kc, ks, k_scale), _values4(vc, vs, v_scale)


# ----------------------------------------------------------------- inputs

def _f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def _table(g, h, need, B):
    """(block_tables, NB): the sequences' pages in a random order of a pool with some to spare."""
    NB, MB = sum(need) + 2 + sum(need) // 8, max(max(need), 1) + 1
    perm = torch.randperm(NB, generator=h).to(torch.int32)
    tables = torch.zeros(len(need), MB, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
    return tables.to(DEV), NB


def _pool4(g, NB, K, B, k_scale, v_scale):
    """A 4-bit pool of normal values, the keys' dims of different sizes, written a piece at a time."""
    cache = torch.empty(NB, K, 144 * B, dtype=torch.uint8, device=DEV)
    dims = (torch.randn(K, 1, D, generator=g, device=DEV) * 0.3).exp()
    t = torch.arange(B, device=DEV)
    each = max(1, (1 << 25) // (K * B * D))
    for at in range(0, NB, each):
        n = min(each, NB - at)
        kc, vc, ks, vs = _sections(cache[at:at + n], B)
        x, s = _quantize4((torch.randn(n, K, B, D, generator=g, device=DEV) * dims).to(torch.bfloat16), k_scale)
        kc.copy_(x)
        ks.copy_(s.view(torch.uint8))
        x, s = _quantize4(torch.randn(n, K, B, D, generator=g, device=DEV).to(torch.bfloat16), v_scale)
        vc.copy_(_swap_halves(x, t))
        vs[..., _scale_place(t[:16])] = s.view(torch.uint8).unflatten(-2, (B // 16, 16)).transpose(-1, -2)
    return cache


def _fp8(g, *shape):
    return (torch.randn(*shape, generator=g, device=DEV) / 0.05).clamp_(-448, 448).to(FP8)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    op, K, B = case["op"], case["kv_heads"], case["block"]
    s = dict(case=case, k_scale=_f32(0.0043), v_scale=_f32(0.0039))
    if op in ("write8", "store4"):
        T = case["tokens"]
        loud = (torch.randn(T, 1, generator=g, device=DEV) * 0.4).exp()     # rows of different sizes
        if case["packed"]:                                          # views of the packed projection of 4 query heads a kv head
            qkv = (torch.randn(T, 6 * K * D, generator=g, device=DEV) * loud).to(torch.bfloat16)
            s["k"], s["v"] = qkv[:, 4 * K * D:5 * K * D].view(T, K, D), qkv[:, 5 * K * D:].view(T, K, D)
        else:
            s["k"], s["v"] = ((torch.randn(T, K * D, generator=g, device=DEV) * loud).to(torch.bfloat16).view(T, K, D)
                              for _ in range(2))
        NB = -(-T // B) + max(1, T // (4 * B)) + 1                  # the last block is no token's
        if case["runs"]:
            blocks = torch.randperm(NB - 1, generator=h)[:-(-T // B)]
            t = torch.arange(T)
            slots = blocks[t // B] * B + t % B
            s["tables"] = blocks[None].to(torch.int32).to(DEV)
        else:
            slots = torch.randperm((NB - 1) * B, generator=h)[:T]
            if op == "write8":
                slots[T - min(case["pad"], T - 1):] = -1            # the padding of a fixed batch
            s["tables"] = (slots // B)[:, None].to(torch.int32).to(DEV)      # each token a sequence of its own
        s["slots"] = slots.to(DEV)
        if op == "store4":
            s["cache"] = _pool4(g, NB, K, B, s["k_scale"], s["v_scale"])
            n = 1 if case["runs"] else T
            s["starts"] = torch.arange(n + 1, dtype=torch.int32, device=DEV) * (T // n)
            s["first"] = None if case["runs"] else (slots % B).to(torch.int32).to(DEV)
        else:
            s["k_cache"], s["v_cache"] = _fp8(g, NB, K, D // 16, B, 16), _fp8(g, NB, K, D, B)
            s["k_scales"], s["v_scales"] = (torch.rand(NB, K, B, generator=g, device=DEV) + 0.01 for _ in range(2))
        return s
    if op == "decode4":
        lens = _lengths(case)
        need = [-(-n // B) for n in lens]
    else:
        spans = _spans(case)
        need = [-(-(f + n) // B) for f, n in spans]
    s["tables"], NB = _table(g, h, need, B)
    if op in ("read4", "decode4"):
        s["cache"] = _pool4(g, NB, K, B, s["k_scale"], s["v_scale"])
    else:
        s["k_cache"] = _fp8(g, NB, K, D // 16, B, 16)
        s["v_cache"] = _fp8(g, NB, K, B // 16, D, 16) if case["shuffled"] else _fp8(g, NB, K, D, B)
        if case["slot"]:
            s["k_scales"], s["v_scales"] = (torch.rand(NB, K, B, generator=g, device=DEV) * 0.02 + 0.002 for _ in range(2))
    if op == "decode4":
        s["q"] = torch.randn(case["seqs"], case["heads"], D, generator=g, device=DEV).to(torch.bfloat16)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["sinks"] = torch.randn(case["heads"], generator=g, device=DEV) + 2 if case["sinks"] else None
        s["scale"], s["max_len"] = D ** -0.5, max(max(lens), 1)
        return s
    starts = torch.tensor([0] + [n for _, n in spans]).cumsum(0)
    s["tokens"] = int(starts[-1]) + case["pad"]
    s["starts"] = starts.to(torch.int32).to(DEV)
    s["first"] = torch.tensor([f for f, _ in spans], dtype=torch.int32, device=DEV)
    s["k_out"], s["v_out"] = (torch.zeros(s["tokens"], K, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    return s


# -------------------------------------------------------------------- run

def run(s):
    op = s["case"]["op"]
    if own:
        import paged_kv_decode_pda_gb300 as pda
        return _own(pda, s, op)
    return {"write8": _plain_write8, "read8": _plain_read8, "store4": _plain_store4, "read4": _plain_read4,
            "decode4": _plain_decode4}[op](s)


def _own(pda, s, op):
    c = s["case"]
    if op == "write8":
        pda.reshape_and_cache_slot_scales(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                          s["slots"], min_scale=MIN_SCALE)
        return s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]
    if op == "store4":
        pda.reshape_and_cache_fp4(s["k"], s["v"], s["cache"], s["slots"], s["k_scale"], s["v_scale"])
        k, v = pda.gather_cache_fp4(s["cache"], s["tables"], s["starts"], c["tokens"], s["k_scale"], s["v_scale"],
                                    first=s["first"])
        return k, v, s["cache"]
    if op == "read8":
        if c["slot"]:
            return pda.gather_cache_slot_scales(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["tables"],
                                                s["starts"], s["tokens"], first=s["first"], k_out=s["k_out"],
                                                v_out=s["v_out"])
        return pda.gather_cache(s["k_cache"], s["v_cache"], s["tables"], s["starts"], s["tokens"], s["k_scale"],
                                s["v_scale"], first=s["first"], v_shuffled=c["shuffled"], k_out=s["k_out"],
                                v_out=s["v_out"])
    if op == "read4":
        return pda.gather_cache_fp4(s["cache"], s["tables"], s["starts"], s["tokens"], s["k_scale"], s["v_scale"],
                                    first=s["first"], k_out=s["k_out"], v_out=s["v_out"])
    return pda.decode_fp4(s["q"], s["cache"], s["tables"], s["lens"], s["scale"], s["k_scale"], s["v_scale"],
                          window=c["window"], sinks=s["sinks"])


def _rows8(x):
    """Rows [..., 128] -> (e4m3 codes, scales [..., 1] in 32 bits)."""
    x = x.float()
    scale = _over(_finite_amax(x), 448.0).clamp(min=MIN_SCALE)
    return _to_e4m3(x.double() / scale.double()), scale


def _plain_write8(s):
    c = s["case"]
    T, K, B = c["tokens"], c["kv_heads"], c["block"]
    k, ks = _rows8(s["k"])
    v, vs = _rows8(s["v"])
    kc, vc = s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8)
    pad = s["slots"] < 0
    slot = torch.where(pad, kc.shape[0] * B - 1, s["slots"])                        # padding rewrites a slot of no token
    b, o = slot // B, slot % B
    pad = pad[:, None, None]
    k, v = k.view(torch.uint8), v.view(torch.uint8)
    kc[b, :, :, o, :] = torch.where(pad, kc[b, :, :, o, :].reshape(T, K, D), k).view(T, K, D // 16, 16)
    vc[b, :, :, o] = torch.where(pad, vc[b, :, :, o], v)
    for table, x in ((s["k_scales"], ks), (s["v_scales"], vs)):
        table[b, :, o] = torch.where(pad[..., 0], table[b, :, o], x[..., 0])
    return s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]


def _rows_of(s, T, starts, first, B, tables):
    """(page, slot in it) of every row of a packed read, and whether the row is a sequence's."""
    r = torch.arange(T, device=DEV)
    of = torch.searchsorted(starts[1:].contiguous(), r, right=True)
    S = tables.shape[0]
    mine = of.clamp(max=S - 1)
    p = r - starts[mine].long()
    if first is not None:
        p = p + first[mine].long()
    p = torch.where(of < S, p, 0)
    return tables[mine, p // B].long(), p % B, (of < S)[:, None, None]


def _plain_store4(s):
    c = s["case"]
    B = c["block"]
    b, o = s["slots"] // B, s["slots"] % B
    kc, vc, ks, vs = _sections(s["cache"], B)
    x, a = _quantize4(s["k"], s["k_scale"])
    kc[b, :, o], ks[b, :, o] = x, a.view(torch.uint8)
    x, a = _quantize4(s["v"], s["v_scale"])
    vc[b, :, o] = _swap_halves(x, o[:, None])
    vs[b, :, o // 16, :, _scale_place(o % 16)] = a.view(torch.uint8)
    k, v, _ = _read4(s, c["tokens"])
    return k.to(torch.bfloat16), v.to(torch.bfloat16), s["cache"]


def _read4(s, T):
    B = s["case"]["block"]
    b, o, mine = _rows_of(s, T, s["starts"], s["first"], B, s["tables"])
    kc, vc, ks, vs = _sections(s["cache"], B)
    k = _values4(kc[b, :, o], ks[b, :, o], s["k_scale"])
    v = _values4(_swap_halves(vc[b, :, o], o[:, None]), vs[b, :, o // 16, :, _scale_place(o % 16)], s["v_scale"])
    return k, v, mine


def _plain_read4(s):
    k, v, mine = _read4(s, s["tokens"])
    for out, x in ((s["k_out"], k), (s["v_out"], v)):
        out.copy_(torch.where(mine, x.to(torch.bfloat16), out))
    return s["k_out"], s["v_out"]


def _plain_read8(s):
    c = s["case"]
    K, B, T = c["kv_heads"], c["block"], s["tokens"]
    b, o, mine = _rows_of(s, T, s["starts"], s["first"], B, s["tables"])
    kc, vc = s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8)
    k = kc[b, :, :, o, :].reshape(T, K, D)
    v = vc[b, :, o // 16, :, o % 16] if c["shuffled"] else vc[b, :, :, o]
    ks, vs = s["k_scale"], s["v_scale"]
    if c["slot"]:
        ks, vs = s["k_scales"][b, :, o][..., None], s["v_scales"][b, :, o][..., None]
    for out, x, scale in ((s["k_out"], k, ks), (s["v_out"], v, vs)):
        out.copy_(torch.where(mine, (x.contiguous().view(FP8).float() * scale).to(torch.bfloat16), out))
    return s["k_out"], s["v_out"]


def _plain_decode4(s):
    c = s["case"]
    S, H, K, B = c["seqs"], c["heads"], c["kv_heads"], c["block"]
    pages = s["tables"][:, :-(-s["max_len"] // B)].long()
    L = pages.shape[1] * B
    k, v = (x.transpose(1, 2).reshape(S, K, L, D) for x in _pages4(s["cache"], pages, B, s["k_scale"], s["v_scale"]))
    t = torch.arange(L, device=DEV)
    n = s["lens"].long()[:, None]
    seen = t < n
    if c["window"]:
        seen = seen & (t >= n - c["window"])
    q = s["q"].float().view(S, K, H // K, D)
    z = (q @ k.transpose(-1, -2)).mul_(s["scale"])
    z = torch.where(seen[:, None, None], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, K, H // K, 1)
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, 0.0, m)
    e = (z - m).exp_()
    total = e.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + (sink - m).exp()
    o = e @ v.masked_fill_(~seen[:, None, :, None], 0.0)
    return torch.where(total > 0, o / total, 0.0).reshape(S, H, D).to(torch.bfloat16)


# ------------------------------------------------------------ 64-bit values

def _nearest(x, grid):
    """Index into the ascending ``grid`` (64 bits, >= 0) next to |x|; a tie goes to the even index."""
    grid = torch.tensor(grid, dtype=torch.float64, device=DEV)
    mid = (grid[1:] + grid[:-1]) / 2
    x = x.abs().contiguous()
    lo = torch.searchsorted(mid, x, right=False)                    # a tie is left below
    hi = torch.searchsorted(mid, x, right=True)                     # a tie is put above
    return torch.where(lo % 2 == 0, lo, hi)


def _grid8():
    """The non-negative e4m3 values in the order of their codes."""
    return [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]


def _exact4(x, scale):
    """Values [..., 128] (64 bits) after the way through 4 bits."""
    grid8, grid4 = (torch.tensor(v, dtype=torch.float64, device=DEV) for v in (_grid8(), E2M1))
    out = torch.empty_like(x)
    for d in range(0, D, 16):
        part = x[..., d:d + 16]
        unit = grid8[_nearest(_over(part.abs().amax(-1), 6.0 * scale), _grid8())][..., None] * scale
        y = torch.where(unit == 0, 0.0, part / torch.where(unit == 0, 1.0, unit))
        out[..., d:d + 16] = grid4[_nearest(y, E2M1)] * torch.sign(part) * unit
    return out


def _exact_values4(record, B, slot, k_scale, v_scale):
    """(K, V) [n, 128] in 64 bits of slots ``slot`` [n] of the records [n, 144 * B], byte by byte from the layout."""
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=DEV)
    d = torch.arange(D, device=DEV)[None]
    t = slot[:, None]

    def at(place):
        return record.gather(1, place.expand(record.shape[0], -1))

    out = []
    for kind, scale in ((0, k_scale), (1, v_scale)):
        byte = d // 2
        if kind:
            byte = byte ^ ((t >> 1 & 1) * 32)
        code = at(64 * B * kind + 64 * t + byte) >> (4 * (d % 2)).to(torch.uint8) & 15
        u = t % 16
        place = 128 * B + 8 * t + d // 16 if not kind else \
            136 * B + (t // 16) * 128 + (d // 16) * 16 + 4 * ((u % 4) ^ (u // 4 % 2)) + u // 4
        out.append(table[code.long()] * at(place).view(FP8).double() * scale)
    return out


def exact(case, seed):
    """What ``run`` returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    op, K, B = case["op"], case["kv_heads"], case["block"]
    if op == "write8":
        at = torch.nonzero(s["slots"] >= 0)[:, 0]
        b, o = s["slots"][at] // B, s["slots"][at] % B
        caches, tables = [], []
        grid = torch.tensor(_grid8(), dtype=torch.float64, device=DEV)
        for name, x in (("k", s["k"]), ("v", s["v"])):
            x = x[at].double()
            scale = _over(x.abs().amax(-1), 448.0).clamp(min=MIN_SCALE)
            held = scale.float().double()                           # the codes are for the scale as it is held
            codes = grid[_nearest(x / held[..., None], _grid8())] * torch.sign(x)
            cache, table = s[name + "_cache"].double(), s[name + "_scales"].double()
            for h in range(K):
                table[b, h, o] = scale[:, h]
                for d in range(D):
                    if name == "k":
                        cache[b, h, d // 16, o, d % 16] = codes[:, h, d]
                    else:
                        cache[b, h, d, o] = codes[:, h, d]
            caches.append(cache)
            tables.append(table)
        return (*caches, *tables)
    if op == "store4":
        return _exact4(s["k"].double(), s["k_scale"]), _exact4(s["v"].double(), s["v_scale"]), None
    if op in ("read8", "read4"):
        k, v = s["k_out"].double(), s["v_out"].double()
        r0 = 0
        for i, (first, n) in enumerate(_spans(case)):
            if not n:
                continue
            pos = torch.arange(first, first + n, device=DEV)
            ids, o = s["tables"][i, pos // B].long(), pos % B
            for h in range(K):
                if op == "read4":
                    k[r0:r0 + n, h], v[r0:r0 + n, h] = _exact_values4(s["cache"][ids, h], B, o, s["k_scale"], s["v_scale"])
                    continue
                kk = s["k_cache"].view(torch.uint8)[ids, h]         # [n, 8, bs, 16]
                vv = s["v_cache"].view(torch.uint8)[ids, h]
                kk = kk[torch.arange(n, device=DEV), :, o].flatten(1).view(FP8).double()
                if case["shuffled"]:
                    vv = vv[torch.arange(n, device=DEV), o // 16, :, o % 16]
                else:
                    vv = vv[torch.arange(n, device=DEV), :, o]
                vv = vv.contiguous().view(FP8).double()
                if case["slot"]:
                    k[r0:r0 + n, h] = kk * s["k_scales"][ids, h, o].double()[:, None]
                    v[r0:r0 + n, h] = vv * s["v_scales"][ids, h, o].double()[:, None]
                else:
                    k[r0:r0 + n, h], v[r0:r0 + n, h] = kk * s["k_scale"], vv * s["v_scale"]
            r0 += n
        return k, v
    H = case["heads"]
    out = torch.zeros(case["seqs"], H, D, dtype=torch.float64, device=DEV)
    for i, n in enumerate(_lengths(case)):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        pos = torch.arange(lo, n, device=DEV)
        ids = s["tables"][i, pos // B].long()
        for h in range(K):
            key, val = _exact_values4(s["cache"][ids, h], B, pos % B, s["k_scale"], s["v_scale"])
            rows = slice(h * (H // K), (h + 1) * (H // K))
            z = s["q"][i, rows].double() @ key.T * s["scale"]
            if s["sinks"] is not None:
                z = torch.cat([z, s["sinks"][rows].double()[:, None]], 1)
            w = torch.softmax(z, 1)
            out[i, rows] = w[:, :n - lo] @ val
    return out
