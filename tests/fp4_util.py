"""Inputs and plain forms, on the CPU in 64 bits, of tests that look at single weights and single pages of a 4-bit cache."""

from __future__ import annotations

import numpy as np
import torch

from tests import lowbits_util as U

ONE = 0x38                                                          # e4m3 1.0


def write_rows(cache, bs, kind, slots, values, scales):
    """Rows of e2m1 values [n, Hk, 128] and group scales [n, Hk, 8] (e4m3 values) at `slots` of a CPU cache."""
    grid = torch.from_numpy(U.E2M1)
    codes = torch.searchsorted(grid, values.abs().double().contiguous()).to(torch.uint8) | ((values < 0).to(torch.uint8) << 3)
    U.write4(cache, bs, kind, slots, codes, scales.to(torch.float8_e4m3fn).view(torch.uint8))


def shuffled_tables(lens, bs, generator, extra=1):
    """(tables [S, MB] of distinct pages in a random order, NB); entries that no token needs name a block of nobody."""
    need = [-(-n // bs) for n in lens]
    NB = sum(need) + 2
    perm = torch.randperm(NB, generator=generator).to(torch.int32)
    tables = torch.full((len(lens), max(need + [1]) + extra), int(perm[-1]), dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
    return tables, NB


# ------------------------------------------------- a far token and small weights

class FarToken:
    """One context that all sequences share. Its first token lies G (log2) in front of the others, which differ among
    themselves, and its V is zero: the small weights alone make the output. G is every (sequence, head)'s own, 0 to 33."""

    ks, vs, scale = 0.125, 0.25, 0.5

    def __init__(self, n, S, H, Hk, bs, seed):
        g = torch.Generator().manual_seed(seed)
        self.n, self.S, self.H, self.Hk, self.bs = n, S, H, Hk, bs
        self.tables, NB = shuffled_tables([n], bs, g)
        self.cache = torch.zeros(NB, Hk, 144 * bs, dtype=torch.uint8)
        pos = torch.arange(n)
        slots = self.tables[0, pos // bs].long() * bs + pos % bs
        grid = torch.from_numpy(U.E2M1)
        self.k = torch.zeros(n, Hk, 128, dtype=torch.float64)
        self.k[:, :, 0] = grid[torch.randint(0, 8, (n, Hk), generator=g)]
        self.k[0, :, 0] = 6
        ks = torch.ones(n, Hk, 8, dtype=torch.float64)
        ks[:, :, 0] = 64.0
        ks[0, :, 0] = 448.0
        write_rows(self.cache, bs, 0, slots, self.k, ks)
        self.key = self.k[:, :, 0] * ks[:, :, 0] * self.ks          # [n, Hk]: dim 0, the only one
        self.v = grid[torch.randint(1, 8, (n, Hk, 128), generator=g)]
        self.v[0] = 0
        write_rows(self.cache, bs, 1, slots, self.v, torch.ones(n, Hk, 8, dtype=torch.float64))
        gaps = torch.rand(S, H, generator=g, dtype=torch.float64) * 33
        self.q = torch.zeros(S, H, 128, dtype=torch.bfloat16)
        self.q[:, :, 0] = (gaps * np.log(2.0) / (6 * 448 * self.ks * self.scale)).to(torch.bfloat16)

    def plain(self, sinks=None, drop=None, weights=None):
        """(out float64 [S, H, 128], tolerance of a bf16 result). `weights`: what becomes of the weights before the product.

        Tolerance, with w the weights relative to the far token's (the largest):
          2^-11 of the weighted mean of |v|   the weights in one f16
          2^-32 n max|v| / sum w              those below f16's normal numbers, off by a fixed amount
          2^-12 of the weighted mean          sums of n <= 2^10 equal-signed terms in binary32, exponents of up to 33 in
                                              binary32 (2^-18), the exponential (2^-22)
          2^-8 |out|                          the output's rounding"""
        G = self.H // self.Hk
        out = torch.empty(self.S, self.H, 128, dtype=torch.float64)
        tol = torch.empty_like(out)
        for h in range(self.H):
            z = self.q[:, h, :1].double() * self.key[:, h // G] * self.scale       # [S, n]
            w = (z - z[:, :1]).exp()
            if drop is not None:
                w[:, drop] = 0
            total = w.sum(1, keepdim=True)
            if sinks is not None:
                total = total + (sinks[h].double() - z[:, :1]).exp()
            val = self.v[:, h // G] * self.vs
            out[:, h] = ((w if weights is None else weights(w)) @ val) / total
            tol[:, h] = out[:, h] * (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -8) + 2.0 ** -32 * self.n * val.max() / total
        return out, tol


# ------------------------------------------------------------ marked pages

class MarkedPages:
    """Contexts of distinct pages with equal weights: page j of a sequence holds ones in the single dim mark(j, kv head) of V,
    zeros elsewhere, so that every output is a count of tokens over the length, and each page is seen in one of them."""

    vs = 0.5

    def __init__(self, lens, H, Hk, bs, seed=0, extra=1, cache=True):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.Hk, self.bs = lens, H, Hk, bs
        self.tables, NB = shuffled_tables(lens, bs, g, extra)
        if not cache:
            return
        self.cache = torch.zeros(NB, Hk, 144 * bs, dtype=torch.uint8)
        codes, shift, scales = U.Record(bs).tables()
        self.cache[..., 128 * bs:] = 0x7F                           # NaN wherever no token lies
        for i, n in enumerate(lens):
            j = torch.arange(-(-n // bs))
            ids = self.tables[i, j].long()
            for o in range(bs):
                here = j * bs + o < n
                for h in range(Hk):
                    rows = self.cache[:, h]
                    rows[ids[here][:, None], scales[:, o].flatten()[None]] = ONE
                    dim = self.mark(j[here], h)
                    rows[ids[here], codes[1, o, dim]] = (2 << shift[dim]).to(torch.uint8)   # e2m1 1.0
        self.q = torch.randn(len(lens), H, 128, generator=g).to(torch.bfloat16)

    @staticmethod
    def mark(j, h):
        return (j * 37 + h * 11) % 128

    def counts(self, i, lo=0, drop=(), twice=()):
        """Tokens [Hk, 128] of sequence i by mark, from position lo on; pages in `drop` left out, in `twice` counted twice."""
        n = self.lens[i]
        j = torch.arange(-(-n // self.bs))
        tokens = (torch.minimum((j + 1) * self.bs, torch.tensor(n)) - torch.clamp(j * self.bs, min=lo)).clamp(min=0)
        tokens[list(drop)] = 0
        tokens[list(twice)] *= 2
        out = torch.zeros(self.Hk, 128, dtype=torch.float64)
        for h in range(self.Hk):
            out[h].index_add_(0, self.mark(j, h), tokens.double())
        return out

    def plain(self, i, window=0, **kw):
        c = self.counts(i, max(0, self.lens[i] - window) if window else 0, **kw)
        n = c.sum(1, keepdim=True)
        return torch.where(n > 0, c / n.clamp(min=1) * self.vs, 0.0)

    @staticmethod
    def agrees(got, want):
        """Where [.., 128] rows agree. The weights are equal and their sums whole multiples of one of them, so what rounds is
        the quotient (2^-16 is ample for a binary32 division and n sums of one binary32 number) and the output (2^-8)."""
        return (got - want).abs() <= want * (2.0 ** -8 + 2.0 ** -16)


MARKED = [([70000], 8, 1, 64, 0), ([70000, 3], 2, 2, 128, 0), ([131072], 4, 4, 16, 0), ([20000, 50, 0, 6000, 1], 5, 1, 32, 0),
          ([60000, 60001], 16, 2, 16, 0), ([33000, 1, 129], 21, 3, 48, 0), ([70000, 40000], 8, 1, 64, 30011),
          ([9000] * 40, 4, 4, 16, 0)]


# ------------------------------------------------------------------ by length

def decode_by_length(q, cache, tables, lens, bs, scale, ks, vs, most=1 << 17):
    """(out float64 [S, H, 128], the weighted means of |v|, max|v| * n) of many short sequences: those of one length together."""
    S, H, _ = q.shape
    Hk = cache.shape[1]
    out, mean, top = (torch.zeros(S, H, 128, dtype=torch.float64) for _ in range(3))
    for n in sorted(set(lens.tolist())):
        if n <= 0:
            continue
        mine = torch.nonzero(lens == n)[:, 0]
        for part in mine.split(max(1, most // (n * Hk))):
            pos = torch.arange(n)
            ids = tables[part][:, pos // bs].long().flatten()
            o = (pos % bs).repeat(len(part))
            k, v = (U.read4(cache, bs, kind, ids, o, s)[1].view(len(part), n, Hk, 128) for kind, s in ((0, ks), (1, vs)))
            qq = q[part].double().view(len(part), Hk, H // Hk, 128)
            w = torch.softmax(torch.einsum("shgd,snhd->shgn", qq, k) * scale, -1)
            out[part] = torch.einsum("shgn,snhd->shgd", w, v).reshape(len(part), H, 128)
            mean[part] = torch.einsum("shgn,snhd->shgd", w, v.abs()).reshape(len(part), H, 128)
            top[part] = n * v.abs().amax((1, 2, 3)).view(-1, 1, 1)
    return out, mean, top
