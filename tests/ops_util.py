"""64-bit plain forms of the operators around the decode call, and inputs for their tests.

Everything here runs on the CPU in float64 / Python integers and shares no
code with the library.
"""

from __future__ import annotations

import math

import numpy as np
import torch

D = 128
FP8 = torch.float8_e4m3fn


def e4m3(*shape, g, scale=0.05):
    return (torch.randn(*shape, generator=g) / scale).clamp(-448, 448).to(FP8)


# ------------------------------------------------------------------- rope

def rope64(x: torch.Tensor, positions: torch.Tensor, inv_freq, magnitude=1.0, interleaved=False) -> torch.Tensor:
    """x [T, heads, D] -> float64, the rotation by its definition."""
    y = x.double().clone()
    n = len(inv_freq)
    for t, p in enumerate(positions.tolist()):
        for i, f in enumerate(inv_freq.tolist()):
            ang = float(p) * float(f)    # off by 2^-53 of the angle: 2e-10 rad at 10^6
            c, s = math.cos(ang) * magnitude, math.sin(ang) * magnitude
            d0, d1 = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            u, v = y[t, :, d0].clone(), y[t, :, d1].clone()
            y[t, :, d0] = u * c - v * s
            y[t, :, d1] = u * s + v * c
    return y


# ----------------------------------------------------------------- extend

class Chunk:
    """One call's inputs on the CPU: sequences of (new, total) tokens over a shuffled pool."""

    def __init__(self, seqs, heads, kv_heads, bs=16, *, seed=0, shuffled=False, pad_front=0, pad_back=0, spare=3,
                 extra_columns=1, garbage=True, q_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.H, self.K, self.bs, self.shuffled = list(seqs), heads, kv_heads, bs, shuffled
        need = [-(-n // bs) for _, n in seqs]
        NB = sum(need) + spare
        MB = max(need + [1]) + extra_columns
        self.NB = NB
        self.k_cache = e4m3(NB, kv_heads, D // 16, bs, 16, g=g)
        vshape = (NB, kv_heads, bs // 16, D, 16) if shuffled else (NB, kv_heads, D, bs)
        self.v_cache = e4m3(*vshape, g=g)
        perm = torch.randperm(NB, generator=g).tolist()
        self.tables = torch.full((len(seqs), MB), perm[-1], dtype=torch.int32)   # unused entries: an unused block
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
            at += n
        if garbage:   # what no token fills is NaN codes
            used = torch.zeros(NB, bs, dtype=torch.bool)
            for s, (_, n) in enumerate(self.seqs):
                for t in range(n):
                    used[self.tables[s, t // bs], t % bs] = True
            kb, vb = self.k_cache.view(torch.uint8), self.v_cache.view(torch.uint8)
            hole = ~used
            kb[hole[:, None, None, :, None].expand_as(kb)] = 0x7F
            if shuffled:
                vb[hole.view(NB, 1, bs // 16, 1, 16).expand_as(vb)] = 0xFF
            else:
                vb[hole[:, None, None, :].expand_as(vb)] = 0xFF
        self.starts = [pad_front]
        for n, _ in self.seqs:
            self.starts.append(self.starts[-1] + n)
        self.T = self.starts[-1] + pad_back
        self.q = (torch.randn(self.T, heads, D, generator=g) * q_scale).to(torch.bfloat16)
        self.lens = [n for _, n in self.seqs]
        self.scale, self.ks, self.vs = D ** -0.5, 0.05, 0.04

    def keys_values(self, s):
        """float64 K, V [len, Hk, D] of sequence s."""
        L = self.lens[s]
        ids = self.tables[s, :-(-L // self.bs)].long()
        k = self.k_cache.view(torch.uint8)[ids].view(FP8).double().permute(0, 3, 1, 2, 4).reshape(-1, self.K, D)[:L] * self.ks
        v = self.v_cache.view(torch.uint8)[ids].view(FP8).double()
        v = v.permute(0, 2, 4, 1, 3) if self.shuffled else v.permute(0, 3, 1, 2)
        return k, v.reshape(-1, self.K, D)[:L] * self.vs

    def exact(self, window=0, sinks=None):
        """(out, spread): float64 [T, H, D], NaN in rows of no sequence; spread = sum of weight * |v|, the size
        that relative errors of the weights act on."""
        out = torch.full((self.T, self.H, D), float("nan"), dtype=torch.float64)
        spread = torch.zeros_like(out)
        for s, (n, L) in enumerate(self.seqs):
            if n == 0:
                continue
            k, v = self.keys_values(s)
            k, v = (x.repeat_interleave(self.H // self.K, 1).permute(1, 0, 2) for x in (k, v))   # [H, L, D]
            rows = slice(self.starts[s], self.starts[s + 1])
            z = self.q[rows].double().permute(1, 0, 2) @ k.transpose(1, 2) * self.scale          # [H, n, L]
            p = torch.arange(L - n, L)[:, None]
            t = torch.arange(L)[None]
            seen = t <= p
            if window:
                seen = seen & (t > p - window)
            z = z.masked_fill(~seen, -math.inf)
            if sinks is not None:
                z = torch.cat([z, sinks.double()[:, None, None].expand(-1, n, 1)], 2)
            m = z.amax(2, keepdim=True) if z.shape[2] else torch.zeros(self.H, n, 1, dtype=torch.float64)
            m = torch.where(torch.isinf(m), 0.0, m)
            e = (z - m).exp()
            tot = e.sum(2, keepdim=True)
            w = torch.where(tot > 0, e / tot.clamp(min=1e-300), 0.0)[:, :, :L]
            out[rows] = (w @ v).permute(1, 0, 2)
            spread[rows] = (w @ v.abs()).permute(1, 0, 2)
        return out, spread

    def to(self, dev):
        f = lambda x: x.to(dev)  # noqa: E731
        return dict(q=f(self.q), k_cache=f(self.k_cache), v_cache=f(self.v_cache), block_tables=f(self.tables),
                    seq_lens=f(torch.tensor(self.lens, dtype=torch.int32)),
                    query_starts=f(torch.tensor(self.starts, dtype=torch.int32)), scale=self.scale, k_scale=self.ks,
                    v_scale=self.vs, v_shuffled=self.shuffled)


# Relative error of a weight allowed to the kernel: the weights enter the
# second product as f16 (half a step: 2^-11); as much again for the logits
# (fp32 sums of 128 products off by at most 128 * 2^-24 of sum |q k| * scale,
# below 2^-12 while that sum stays under 32), the exponential and the fp32 sums.
WEIGHT_ERR = 2.0 ** -10


def check_rows(got: torch.Tensor, exact: torch.Tensor, spread: torch.Tensor, label=""):
    """bf16 output against float64: half a bf16 step (2^-8 relative) of the value, and WEIGHT_ERR of the spread."""
    got = got.double().cpu()
    mine = ~torch.isnan(exact[:, 0, 0])
    g, e, s = got[mine], exact[mine], spread[mine]
    assert torch.isfinite(g).all(), "%s: non-finite output" % label
    bound = 2.0 ** -8 * e.abs() + (1 + 2.0 ** -8) * WEIGHT_ERR * s + 1e-30
    worst = ((g - e).abs() / bound).max().item() if g.numel() else 0.0
    assert worst <= 1.0, "%s: %.2f times the bound" % (label, worst)
    return worst


# ------------------------------------------------------------------ pages

class Pool:
    """The page bookkeeping in plain Python: the reference for grow, fork, free and compact."""

    def __init__(self, num_blocks, rows, columns, bs):
        self.refs, self.bs, self.columns = [0] * num_blocks, bs, columns
        self.tables = [[-7] * columns for _ in range(rows)]
        self.lens = [0] * rows
        self.moves = []            # (src, dst) copies of the last call
        self.refused = 0

    def pages(self, n):
        return -(-n // self.bs)

    def free_ids(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def grow(self, rows, add):
        self.refused, self.moves = 0, []
        free, at, seen, todo = self.free_ids(), 0, set(), []
        for r, a in zip(rows, add):
            if r < 0:
                continue
            if r >= len(self.lens) or r in seen:
                self.refused += 1
                continue
            seen.add(r)
            if a < 0 or self.lens[r] + a > self.columns * self.bs:
                self.refused += 1
                continue
            old, new = self.pages(self.lens[r]), self.pages(self.lens[r] + a)
            if new > old and at + new - old > len(free):
                self.refused += 1
            else:
                todo.append((r, a, old, free[at:at + new - old]))
            at += new - old
        for r, a, old, ids in todo:
            for j, i in enumerate(ids):
                self.tables[r][old + j] = i
                self.refs[i] = 1
            self.lens[r] += a

    def fork(self, parents, children):
        self.refused, self.moves = 0, []
        free, at, seen, todo = self.free_ids(), 0, set(), []
        named = {c for p, c in zip(parents, children) if 0 <= c < len(self.lens)}
        for p, c in zip(parents, children):
            if p < 0 or c < 0:
                continue
            if c < len(self.lens) and c not in seen:
                first = True
                seen.add(c)
            else:
                first = False
            if p >= len(self.lens) or not first or p in named or self.lens[c] != 0:
                self.refused += 1
                continue
            part = self.lens[p] % self.bs != 0
            if part and at + 1 > len(free):
                self.refused += 1
            else:
                todo.append((p, c, free[at] if part else None))
            at += part
        for p, c, fresh in todo:
            full = self.lens[p] // self.bs
            for j in range(full):
                i = self.tables[p][j]
                self.tables[c][j] = i
                self.refs[i] += 1
            if fresh is not None:
                self.moves.append((self.tables[p][full], fresh))
                self.tables[c][full] = fresh
                self.refs[fresh] = 1
            self.lens[c] = self.lens[p]

    def free(self, rows):
        self.refused, self.moves = 0, []
        for r in rows:
            if r < 0:
                continue
            if r >= len(self.lens):
                self.refused += 1
                continue
            for j in range(self.pages(self.lens[r])):
                self.refs[self.tables[r][j]] -= 1
            self.lens[r] = 0

    def compact(self):
        self.refused = 0
        live = sum(1 for r in self.refs if r > 0)
        holes = [i for i in range(live) if self.refs[i] == 0]
        movers = [i for i in range(live, len(self.refs)) if self.refs[i] > 0]
        assert len(holes) == len(movers)
        self.moves = list(zip(movers, holes))
        to = dict(self.moves)
        for src, dst in self.moves:
            self.refs[dst], self.refs[src] = self.refs[src], 0
        for r, n in enumerate(self.lens):
            for j in range(self.pages(n)):
                self.tables[r][j] = to.get(self.tables[r][j], self.tables[r][j])

    def tensors(self, dev):
        i32 = torch.int32
        return (torch.tensor(self.refs, dtype=i32, device=dev), torch.tensor(self.tables, dtype=i32, device=dev),
                torch.tensor(self.lens, dtype=i32, device=dev))

    def apply_moves(self, cache: np.ndarray):
        rows = [(s, d, cache[s].copy()) for s, d in self.moves]
        for _, d, page in rows:
            cache[d] = page
