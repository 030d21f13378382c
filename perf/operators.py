"""Cases of the operators around the paged fp8 cache: rotary positions (alone and with the cache write), attention of a
chunk of new tokens, and the pages' bookkeeping with their copies.

``run`` makes one pass: in plain torch operations where ``own`` is false, through the package's calls where it is true.
"""

from __future__ import annotations

import math
import random

import torch

own = False

D = 128
FP8 = torch.float8_e4m3fn
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step's new tokens: 16 sequences, one token each; latency
        dict(name="rope-step-16", op="rope", tokens=16, heads=32, kv_heads=8, rot=128, interleaved=False,
             scaling="none", max_pos=1024),
        # a prefill's tokens out of the packed projection, far positions on a stretched context
        dict(name="rope-prefill-16384", op="rope", tokens=16384, heads=40, kv_heads=8, rot=128, interleaved=False,
             scaling="ramp", max_pos=131072),
        # a padded decode batch: 256 rows, rotated and written at scattered slots
        dict(name="rope_cache-step-256", op="rope_cache", tokens=256, heads=32, kv_heads=8, rot=128, interleaved=True,
             scaling="none", max_pos=4096, block=16, pad=19, runs=False, shuffled=False),
        # a prefill of whole blocks, part of the head rotated
        dict(name="rope_cache-prefill-8192", op="rope_cache", tokens=8192, heads=64, kv_heads=8, rot=64,
             interleaved=False, scaling="bands", max_pos=65536, block=64, pad=0, runs=True, shuffled=False),
        # a short prompt's continuation: one sequence, the smallest call
        dict(name="extend-one-16-of-512", op="extend", seqs=1, new=16, new_lo=16, ctx=512, ctx_lo=512, heads=32,
             kv_heads=8, block=16, window=0, sinks=False, shuffled=False, pad=0, shape=1),
        # checking drafted tokens: 64 sequences of 4 new tokens over ragged contexts
        dict(name="extend-draft-64x4", op="extend", seqs=64, new=4, new_lo=4, ctx=4000, ctx_lo=2000, heads=40,
             kv_heads=8, block=16, window=0, sinks=False, shuffled=False, pad=0, shape=2),
        # chunks of long prompts: 2048 new tokens at the end of 8192
        dict(name="extend-chunk-2x2048-of-8192", op="extend", seqs=2, new=2048, new_lo=2048, ctx=8192, ctx_lo=8192,
             heads=32, kv_heads=8, block=16, window=0, sinks=False, shuffled=False, pad=0, shape=3),
        # a served batch: single tokens and odd chunks mixed, 64-token blocks, sinks and a window, padded rows
        dict(name="extend-mixed-24", op="extend", seqs=24, new=511, new_lo=0, ctx=2048, ctx_lo=0, heads=64, kv_heads=8,
             block=64, window=1024, sinks=True, shuffled=False, pad=13, shape=4),
        # one step of a small beam: drop, fork, grow; latency
        dict(name="branch-8", op="branch", rows=8, drop=2, forks=4, step=1, ctx=1000, kv_heads=8, block=16, arrays=2,
             pool=1024, shape=5),
        # many samples of many prompts, several layers
        dict(name="branch-128", op="branch", rows=128, drop=20, forks=128, step=7, ctx=1024, kv_heads=8, block=64,
             arrays=8, pool=2048, shape=6),
        # a small pool made dense
        dict(name="compact-512", op="compact", pool=512, live=300, rows=12, kv_heads=8, block=16, arrays=2),
        # a pool of several layers, half in use
        dict(name="compact-4096", op="compact", pool=4096, live=2048, rows=64, kv_heads=8, block=16, arrays=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "rope_cache", "extend", "extend", "branch", "compact"))
    kv = rng.choice((1, 2, 4, 8))
    g = rng.choice((1, 2, 3, 4, 5, 7, 8))
    if op in ("rope", "rope_cache"):
        c = dict(op=op, tokens=_log(rng, 1, 12000), heads=kv * g, kv_heads=kv, rot=rng.choice((128, 128, 96, 64, 32, 20)),
                 interleaved=rng.random() < 0.5, scaling=rng.choice(("none", "linear", "base", "ramp", "bands")),
                 max_pos=_log(rng, 64, 1000000))
        if op == "rope_cache":
            runs = rng.random() < 0.5
            c.update(block=rng.choice((16, 32, 48, 64, 128)), pad=0 if runs else _log(rng, 1, 40) - 1, runs=runs,
                     shuffled=rng.random() < 0.3)
        return c
    if op == "extend":
        new = _log(rng, 1, 2048)
        ctx = max(new, _log(rng, 16, 8192))
        room = (2 * 32 * 2048 * 8192) // (kv * g * new * ctx)       # no more than the largest listed case
        seqs = _log(rng, 1, max(1, min(64, room)))
        same = rng.random() < 0.4
        return dict(op=op, seqs=seqs, new=new, new_lo=new if same else 0, ctx=ctx, ctx_lo=ctx if same else 0,
                    heads=kv * g, kv_heads=kv, block=rng.choice((16, 16, 32, 48, 64, 128)),
                    window=rng.choice((0, 0, 1, _log(rng, 2, 4096))), sinks=rng.random() < 0.3,
                    shuffled=rng.random() < 0.25, pad=rng.choice((0, 0, 5)), shape=rng.randrange(1 << 20))
    if op == "branch":
        rows = _log(rng, 1, 128)
        block = rng.choice((16, 32, 64))
        ctx = _log(rng, 8, 1024)
        forks = _log(rng, 1, 128)
        pool = (rows + forks) * ((ctx + 40) // block + 2) + rng.randrange(50)
        arrays = min(rng.choice((1, 2, 4, 8)), max(1, (1 << 30) // (pool * kv * D * block)))
        return dict(op=op, rows=rows, drop=rng.randrange(rows), forks=forks, step=_log(rng, 1, 40), ctx=ctx, kv_heads=kv,
                    block=block, arrays=arrays, pool=pool, shape=rng.randrange(1 << 20))
    pool = _log(rng, 16, 4096)
    block = rng.choice((16, 16, 32))
    arrays = min(rng.choice((1, 2, 8, 16)), max(1, (1 << 30) // (pool * kv * D * block)))
    return dict(op=op, pool=pool, live=_log(rng, 1, pool), rows=_log(rng, 1, 64), kv_heads=kv, block=block, arrays=arrays)


def _lengths(case):
    """(new, total) tokens of each sequence, from the case alone."""
    rng = random.Random(case["shape"])
    out = []
    for _ in range(case["seqs"]):
        n = rng.randint(case["new_lo"], case["new"])
        if case["new_lo"] != case["new"] and rng.random() < 0.4:
            n = min(1, n)                                           # a decoding sequence among the chunks
        out.append((n, max(n, rng.randint(case["ctx_lo"], case["ctx"]))))
    if not any(n for n, _ in out):
        out[0] = (1, max(1, out[0][1]))
    return out


def _row_lengths(case):
    rng = random.Random(case["shape"])
    return [rng.randint(1, case["ctx"]) for _ in range(case["rows"])]


def _page_bytes(case):
    return case["kv_heads"] * D * case["block"]


def work(case):
    op = case["op"]
    if op in ("rope", "rope_cache"):
        T, H, K = case["tokens"], case["heads"], case["kv_heads"]
        rotated = T * (H + K) * (case["rot"] // 2) * 6
        if op == "rope":
            return {"bytes": T * (H + K) * D * 2 * 2 + 8 * T, "flops": rotated}
        w = T - min(case["pad"], T - 1)
        return {"bytes": T * H * D * 4 + w * K * D * 2 * 3 + 16 * T, "flops": rotated + 2 * w * K * D}
    if op == "extend":
        kv_bytes = flops = rows = pages = 0
        for n, length in _lengths(case):
            rows += n
            if n == 0:
                continue
            win = case["window"]
            first = length - n                                      # position of the first new token
            lo = max(0, first - win + 1) if win else 0
            kv_bytes += (length - lo) * case["kv_heads"] * 2 * D
            pages += -(-length // case["block"]) - lo // case["block"]
            if win:
                seen = sum(min(p + 1, win) for p in range(first, length))
            else:
                seen = n * first + n * (n + 1) // 2
            flops += seen * case["heads"] * 4 * D
        return {"bytes": kv_bytes + rows * case["heads"] * D * 4 + 4 * pages + 8 * case["seqs"], "flops": flops}
    if op == "branch":
        S, MB = _table_shape(case)
        copied = case["forks"] * (1 - 1 / case["block"])            # about one partial page a fork
        return {"bytes": 2 * copied * _page_bytes(case) * case["arrays"] + 8 * case["pool"] + 8 * S * MB, "flops": 0}
    moved = case["live"] * (case["pool"] - case["live"]) / case["pool"]
    return {"bytes": 2 * moved * _page_bytes(case) * case["arrays"] + 8 * (case["pool"] + case["live"]), "flops": 0}


# ----------------------------------------------------------------- inputs

def _frequencies(case):
    """Radians per position of each pair (64 bits), and the magnitude, for each way of stretching a context."""
    R, base, s = case["rot"], 10000.0, 8.0
    orig = max(32.0, case["max_pos"] / s)
    kind, mag = case["scaling"], 1.0
    if kind == "base":
        base *= s ** (R / (R - 2.0))
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if kind == "linear":
        f = [x / s for x in f]
    elif kind == "ramp":                                            # by the turns a pair makes over the first context
        def at(turns):
            return R * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(at(32.0))), min(R - 1, math.ceil(at(1.0)))
        keep = [1 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(R // 2)]
        f = [x * k + x / s * (1 - k) for x, k in zip(f, keep)]
        mag = 0.1 * math.log(s) + 1.0
    elif kind == "bands":                                           # by wavelength: short ones kept, long ones stretched
        def band(x):
            wave = 2 * math.pi / x
            if wave < orig / 4:
                return x
            if wave > orig:
                return x / s
            t = (orig / wave - 1) / 3
            return (1 - t) * x / s + t * x
        f = [band(x) for x in f]
    return torch.tensor(f, dtype=torch.float64), mag


def _fp8(g, *shape):
    return (torch.randn(*shape, generator=g, device=DEV) / 0.05).clamp_(-448, 448).to(FP8)


def _table_shape(case):
    return case["rows"] + case["forks"], (case["ctx"] + case["step"]) // case["block"] + 2


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op in ("rope", "rope_cache"):
        T, H, K = case["tokens"], case["heads"], case["kv_heads"]
        qkv = torch.randn(T, (H + 2 * K) * D, generator=g, device=DEV).to(torch.bfloat16)
        s["q"] = qkv[:, :H * D].view(T, H, D)                       # views of the packed projection
        s["k"] = qkv[:, H * D:(H + K) * D].view(T, K, D)
        s["v"] = qkv[:, (H + K) * D:].view(T, K, D)
        s["positions"] = torch.randint(0, case["max_pos"], (T,), generator=g, device=DEV)
        s["inv_freq"], s["magnitude"] = _frequencies(case)
        if op == "rope_cache":
            B = case["block"]
            NB = -(-T // B) + max(1, T // (4 * B)) + 1              # the last block is no token's
            if case["runs"]:
                blocks = torch.randperm(NB - 1, generator=h)[:-(-T // B)]
                t = torch.arange(T)
                slots = blocks[t // B] * B + t % B
            else:
                slots = torch.randperm((NB - 1) * B, generator=h)[:T]
                slots[T - min(case["pad"], T - 1):] = -1            # the padding of a fixed batch
            s["slots"] = slots.to(DEV)
            s["k_cache"] = _fp8(g, NB, K, D // 16, B, 16)
            s["v_cache"] = _fp8(g, NB, K, B // 16, D, 16) if case["shuffled"] else _fp8(g, NB, K, D, B)
            s["k_scale"], s["v_scale"] = 0.05, 0.04
    elif op == "extend":
        H, K, B = case["heads"], case["kv_heads"], case["block"]
        lens = _lengths(case)
        need = [-(-n // B) for _, n in lens]
        NB, MB = sum(need) + 1 + sum(need) // 8, max(max(need), 1) + 1
        perm = torch.randperm(NB, generator=h).to(torch.int32)
        tables = torch.zeros(len(lens), MB, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            tables[i, :n] = perm[at:at + n]
            at += n
        starts = torch.tensor([0] + [n for n, _ in lens]).cumsum(0)
        T = int(starts[-1]) + case["pad"]
        s["q"] = torch.randn(T, H, D, generator=g, device=DEV).to(torch.bfloat16)
        s["k_cache"] = _fp8(g, NB, K, D // 16, B, 16)
        s["v_cache"] = _fp8(g, NB, K, B // 16, D, 16) if case["shuffled"] else _fp8(g, NB, K, D, B)
        s["block_tables"] = tables.to(DEV)
        s["seq_lens"] = torch.tensor([n for _, n in lens], dtype=torch.int32, device=DEV)
        s["starts"] = starts.to(torch.int32).to(DEV)
        s["sinks"] = torch.randn(H, generator=g, device=DEV) + 2 if case["sinks"] else None
        s["max_new"], s["max_len"] = max(n for n, _ in lens), max(n for _, n in lens)
        s["scale"], s["k_scale"], s["v_scale"] = D ** -0.5, 0.05, 0.05
        s["out"] = torch.zeros_like(s["q"])
    elif op == "branch":
        S, MB = _table_shape(case)
        NB, B = case["pool"], case["block"]
        tables, refs, lens = torch.zeros(S, MB, dtype=torch.int32), torch.zeros(NB, dtype=torch.int32), torch.zeros(S, dtype=torch.int32)
        perm, at = torch.randperm(NB, generator=h).to(torch.int32), 0
        for r, n in enumerate(_row_lengths(case)):
            lens[r], pages = n, -(-n // B)
            shared = min(pages, int(lens[r - 1]) // B, n // B) // 2 if r % 2 else 0   # odd rows share a prompt's pages
            if shared:
                tables[r, :shared] = tables[r - 1, :shared]
            tables[r, shared:pages] = perm[at:at + pages - shared]
            at += pages - shared
            refs[tables[r, :pages].long()] += 1
        order = torch.randperm(case["rows"], generator=h)
        keep = order[case["drop"]:]
        parents = keep[torch.randint(0, len(keep), (case["forks"],), generator=h)]
        children = torch.arange(case["rows"], S)
        grown = torch.cat([keep, children])
        s["book"] = torch.cat([refs, lens, tables.view(-1)]).to(DEV)
        for name, x in dict(dropped=order[:case["drop"]], parents=parents, children=children, grown=grown).items():
            s[name] = x.to(torch.int32).to(DEV)
        s["add"] = torch.full((len(grown),), case["step"], dtype=torch.int32, device=DEV)
        s["shape"] = (NB, S, MB)
        s["caches"] = torch.randint(0, 256, (case["arrays"], NB, _page_bytes(case)), generator=g, device=DEV, dtype=torch.uint8)
    else:
        NB, R = case["pool"], case["rows"]
        ids = torch.randperm(NB, generator=h)[:case["live"]].to(torch.int32)
        R = min(R, case["live"])
        cut = sorted(random.Random(case["live"]).sample(range(1, case["live"]), R - 1))   # the rows' pages, from the case alone
        rows = [ids[a:b] for a, b in zip([0] + cut, cut + [case["live"]])]
        MB = max(len(r) for r in rows) + 1
        tables, refs = torch.zeros(R, MB, dtype=torch.int32), torch.zeros(NB, dtype=torch.int32)
        for i, r in enumerate(rows):
            tables[i, :len(r)] = r
            refs[r.long()] = 1 + i % 3 // 2                         # some pages are held from elsewhere too
        lens = torch.tensor([len(r) * case["block"] - 3 for r in rows], dtype=torch.int32)
        s["book"] = torch.cat([refs, lens, tables.view(-1)]).to(DEV)
        s["shape"] = (NB, R, MB)
        s["caches"] = torch.randint(0, 256, (case["arrays"], NB, _page_bytes(case)), generator=g, device=DEV, dtype=torch.uint8)
    return s


def _parts(s, book):
    NB, S, MB = s["shape"]
    return book[:NB], book[NB + S:].view(S, MB), book[NB:NB + S]


# -------------------------------------------------------------------- run

def run(s):
    op = s["case"]["op"]
    if own:
        import paged_kv_decode_pda_gb300 as pda
        return _own(pda, s, op)
    return {"rope": _plain_rope, "rope_cache": _plain_rope_cache, "extend": _plain_extend, "branch": _plain_branch,
            "compact": _plain_compact}[op](s)


def _own(pda, s, op):
    c = s["case"]
    if op == "rope":
        return pda.rope(s["q"], s["k"], s["positions"], s["inv_freq"], magnitude=s["magnitude"],
                        interleaved=c["interleaved"])
    if op == "rope_cache":
        q = pda.rope_and_cache(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"], s["k_cache"],
                               s["v_cache"], s["k_scale"], s["v_scale"], magnitude=s["magnitude"],
                               interleaved=c["interleaved"], v_shuffled=c["shuffled"])
        return q, s["k_cache"], s["v_cache"]
    if op == "extend":
        return pda.extend(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["seq_lens"], s["starts"], s["scale"],
                          s["k_scale"], s["v_scale"], window=c["window"], sinks=s["sinks"], v_shuffled=c["shuffled"],
                          out=s["out"])
    book = s["book"].clone()                                        # the state to come back to is kept
    refs, tables, lens = _parts(s, book)
    caches = s["caches"].unbind(0)
    if op == "branch":
        pda.free_pages(refs, tables, lens, s["dropped"], c["block"])
        pda.fork_pages(refs, tables, lens, s["parents"], s["children"], c["block"], caches)
        pda.grow_pages(refs, tables, lens, s["grown"], s["add"], c["block"])
    else:
        pda.compact_pages(refs, tables, lens, c["block"], caches)
    return book, s["caches"]


def _plain_rotate(x, s):
    c, R = s["case"], s["case"]["rot"]
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].to(DEV)          # [T, 1, R/2]
    cos, sin = (angle.cos() * s["magnitude"]).float(), (angle.sin() * s["magnitude"]).float()
    x = x.float()
    if c["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., R:]], -1)


def _plain_rope(s):
    return _plain_rotate(s["q"], s).to(torch.bfloat16), _plain_rotate(s["k"], s).to(torch.bfloat16)


def _plain_rope_cache(s):
    c, T, K = s["case"], s["case"]["tokens"], s["case"]["kv_heads"]
    q = _plain_rotate(s["q"], s).to(torch.bfloat16)
    k = (_plain_rotate(s["k"], s) / s["k_scale"]).clamp(-448, 448).to(FP8).view(torch.uint8)
    v = (s["v"].float() / s["v_scale"]).clamp(-448, 448).to(FP8).view(torch.uint8)
    kc, vc, B = s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8), c["block"]
    pad = (s["slots"] < 0)[:, None, None]
    slot = torch.where(s["slots"] < 0, kc.shape[0] * B - 1, s["slots"])             # padding rewrites a slot of no token
    b, o = slot // B, slot % B
    k = torch.where(pad, kc[b, :, :, o, :].reshape(T, K, D), k)
    kc[b, :, :, o, :] = k.view(T, K, D // 16, 16)
    if c["shuffled"]:
        vc[b, :, o // 16, :, o % 16] = torch.where(pad, vc[b, :, o // 16, :, o % 16], v)
    else:
        vc[b, :, :, o] = torch.where(pad, vc[b, :, :, o], v)
    return q, s["k_cache"], s["v_cache"]


def _plain_extend(s):
    c = s["case"]
    q, starts, lens = s["q"], s["starts"].long(), s["seq_lens"].long()
    T, H, _ = q.shape
    K, B, S = c["kv_heads"], c["block"], c["seqs"]
    g, N = H // K, s["max_new"]
    pages = s["block_tables"][:, :max(1, -(-s["max_len"] // B))].long()
    L = pages.shape[1] * B
    t = torch.arange(L, device=DEV)
    k = s["k_cache"].view(torch.uint8)[pages].view(FP8).float().permute(0, 2, 1, 4, 3, 5).reshape(S, K, L, D)
    v = s["v_cache"].view(torch.uint8)[pages].view(FP8).float()
    v = v.permute(0, 2, 1, 3, 5, 4) if c["shuffled"] else v.permute(0, 2, 1, 4, 3)
    v = v.reshape(S, K, L, D)
    v = torch.where((t < lens[:, None])[:, None, :, None], v, 0.0)
    i = torch.arange(N, device=DEV)
    rows = (starts[:-1, None] + i).clamp(max=T - 1)
    qp = q[rows].float().view(S, N, K, g, D).permute(0, 2, 3, 1, 4).reshape(S, K, g * N, D)
    z = (qp @ k.transpose(-1, -2)).mul_(s["scale"] * s["k_scale"]).view(S, K, g, N, L)
    new = starts[1:] - starts[:-1]
    p = (lens - new)[:, None, None] + i[:, None]                                    # [S, N, 1]
    seen = t <= p
    if c["window"]:
        seen = seen & (t > p - c["window"])
    z = torch.where(seen[:, None, None], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, K, g, 1, 1)
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, 0.0, m)
    e = (z - m).exp_()
    total = e.sum(-1, keepdim=True)
    o = (e.view(S, K, g * N, L) @ v).view(S, K, g, N, D)
    if s["sinks"] is not None:
        total = total + (sink - m).exp()
    o = torch.where(total > 0, o / total * s["v_scale"], 0.0).permute(0, 3, 1, 2, 4).reshape(S, N, H, D)
    r = torch.arange(T, device=DEV)
    of = torch.searchsorted(starts[1:].contiguous(), r, right=True)
    mine = of.clamp(max=S - 1)
    o = o[mine, (r - starts[mine]).clamp(0, N - 1)].to(torch.bfloat16)
    s["out"].copy_(torch.where((of < S)[:, None, None], o, s["out"]))
    return s["out"]


def _plain_free_list(refs):
    """The ids of the free pages, lowest first (the rest of the list is of no use)."""
    free = refs == 0
    n = refs.numel()
    to = torch.where(free, free.cumsum(0) - 1, n)
    return torch.zeros(n + 1, dtype=torch.int64, device=DEV).scatter_(0, to, torch.arange(n, device=DEV))


def _plain_branch(s):
    c, B = s["case"], s["case"]["block"]
    book = s["book"].clone()
    refs, tables, lens = _parts(s, book)
    S, MB = tables.shape
    j = torch.arange(MB, device=DEV)
    # free
    d = s["dropped"].long()
    held = j < ((lens[d] + B - 1) // B)[:, None]
    refs.scatter_add_(0, torch.where(held, tables[d], 0).long().view(-1), -held.view(-1).to(torch.int32))
    lens[d] = 0
    # fork
    p, ch = s["parents"].long(), s["children"].long()
    L = lens[p]
    full, part = L // B, L % B != 0
    fresh = _plain_free_list(refs)[(part.cumsum(0) - 1).clamp(min=0)].to(torch.int32)
    row = tables[p]
    src = torch.where(part, row.gather(1, full.long()[:, None].clamp(max=MB - 1))[:, 0], row[:, 0])
    row = torch.where(part[:, None] & (j == full[:, None]), fresh[:, None], row)
    held = j < full[:, None]
    refs.scatter_add_(0, torch.where(held, row, 0).long().view(-1), held.view(-1).to(torch.int32))
    refs.scatter_add_(0, torch.where(part, fresh, 0).long(), part.to(torch.int32))
    tables[ch] = torch.where(j < ((L + B - 1) // B)[:, None], row, tables[ch])
    lens[ch] = L
    dst = torch.where(part, fresh, src).long()
    s["caches"][:, dst] = s["caches"][:, src.long()]
    # grow
    r = s["grown"].long()
    old, new = (lens[r] + B - 1) // B, (lens[r] + s["add"] + B - 1) // B
    need = new - old
    at = (need.cumsum(0) - need)[:, None] + j - old[:, None]
    more = (j >= old[:, None]) & (j < new[:, None])
    ids = _plain_free_list(refs)[torch.where(more, at, 0)].to(torch.int32)
    tables[r] = torch.where(more, ids, tables[r])
    refs.scatter_add_(0, torch.where(more, ids, 0).long().view(-1), more.view(-1).to(torch.int32))
    lens[r] += s["add"]
    return book, s["caches"]


def _plain_compact(s):
    B = s["case"]["block"]
    book = s["book"].clone()
    refs, tables, lens = _parts(s, book)
    n = refs.numel()
    ids = torch.arange(n, device=DEV)
    live = refs > 0
    count = live.sum()
    hole = torch.nonzero(~live & (ids < count))[:, 0]
    mover = torch.nonzero(live & (ids >= count))[:, 0]
    to = ids.clone()
    to[mover] = hole
    held = torch.arange(tables.shape[1], device=DEV) < ((lens + B - 1) // B)[:, None]
    tables.copy_(torch.where(held, to[torch.where(held, tables, 0).long()].to(torch.int32), tables))
    refs[hole] = refs[mover]
    refs[mover] = 0
    s["caches"][:, hole] = s["caches"][:, mover]
    return book, s["caches"]


# ------------------------------------------------------------ 64-bit values

def exact(case, seed):
    """The floating outputs from their definitions in 64 bits; the pages' cases are whole numbers throughout."""
    op = case["op"]
    if op in ("branch", "compact"):
        return None
    s = prepare(case, seed)
    if op == "extend":
        return _exact_extend(case, s)
    H, R = case["heads"], case["rot"]
    theta = torch.outer(s["positions"].double(), s["inv_freq"].to(DEV))

    def turned(x):
        y = x.double().clone()
        first = torch.arange(R // 2, device=DEV) * 2 if case["interleaved"] else torch.arange(R // 2, device=DEV)
        second = first + 1 if case["interleaved"] else first + R // 2
        z = torch.polar(torch.full_like(theta, s["magnitude"]), theta)[:, None] * torch.complex(y[..., first], y[..., second])
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k = turned(s["q"]), turned(s["k"])
    if op == "rope":
        return q, k
    B = case["block"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    at = torch.nonzero(s["slots"] >= 0)[:, 0]
    b, o = s["slots"][at] // B, s["slots"][at] % B
    kq, vq = ((x / y).clamp(-448, 448)[at] for x, y in ((k, s["k_scale"]), (s["v"].double(), s["v_scale"])))
    for h in range(case["kv_heads"]):
        for d in range(D):
            kc[b, h, d // 16, o, d % 16] = kq[:, h, d]
            if case["shuffled"]:
                vc[b, h, o // 16, d, o % 16] = vq[:, h, d]
            else:
                vc[b, h, d, o] = vq[:, h, d]
    return q, kc, vc


def _exact_extend(case, s):
    H, K, B = case["heads"], case["kv_heads"], case["block"]
    out = s["out"].double()
    r0 = 0
    for i, (n, length) in enumerate(_lengths(case)):
        if n:
            ids = s["block_tables"][i, :-(-length // B)].long()
            kk = s["k_cache"][ids].double() * s["k_scale"]
            vv = s["v_cache"][ids].double() * s["v_scale"]
            pos = torch.arange(length - n, length, device=DEV)[:, None]
            t = torch.arange(length, device=DEV)[None]
            hidden = t > pos
            if case["window"]:
                hidden = hidden | (t <= pos - case["window"])
            for h in range(H):
                kv = h // (H // K)
                key = kk[:, kv].transpose(1, 2).reshape(-1, D)[:length]             # [pages, bs, D/16, 16]
                val = vv[:, kv].transpose(2, 3) if case["shuffled"] else vv[:, kv].transpose(1, 2)
                val = val.reshape(-1, D)[:length]
                z = (s["q"][r0:r0 + n, h].double() @ key.T * s["scale"]).masked_fill_(hidden, -math.inf)
                if s["sinks"] is not None:
                    z = torch.cat([z, s["sinks"][h].double().expand(n, 1)], 1)
                w = z.sub_(z.amax(1, keepdim=True)).exp_()
                w /= w.sum(1, keepdim=True)
                out[r0:r0 + n, h] = w[:, :length] @ val
        r0 += n
    return out
