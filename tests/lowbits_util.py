"""64-bit plain forms of the caches in fewer bits, on the CPU, sharing no code with the library.

A rounding decision compares |x| with midpoint * scale, a product that binary64
holds exactly (5 + 24 + 4 bits), so every code here is the one that the real
quotient rounds to.
"""

from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])   # by code, 0 .. 448


def nearest_code(ax: np.ndarray, unit: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Code of the grid value nearest to ax / unit (ax >= 0, unit > 0); ties to the even code; past the end, the last."""
    code = np.zeros(ax.shape, dtype=np.int64)
    for i in range(len(grid) - 1):
        edge = (grid[i] + grid[i + 1]) / 2 * unit
        code += (ax > edge) | ((ax == edge) & ((i + 1) % 2 == 0))
    return code


def _finite_amax(x):
    return np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)


def quantize_rows8(x: torch.Tensor, min_scale: float):
    """Rows [..., 128] -> (e4m3 bytes uint8 [..., 128], scales float32 [...])."""
    x = x.double().numpy()
    scale = np.maximum((_finite_amax(x) / 448.0).astype(np.float32), np.float32(min_scale))
    big = np.where(np.isnan(x), 0.0, np.abs(x))
    code = nearest_code(np.minimum(big, 1e300), np.broadcast_to(scale.astype(np.float64)[..., None], x.shape), E4M3)
    code = np.where(np.isnan(x), 0x7F, code | (np.signbit(x).astype(np.int64) << 7))
    return torch.from_numpy(code.astype(np.uint8)), torch.from_numpy(scale)


def quantize_rows4(x: torch.Tensor, g: float):
    """Rows [..., 128] -> (codes uint8 [..., 128] of 4 bits, group scales e4m3 bytes [..., 8]). NaN groups: codes 0."""
    g = float(np.float32(g))
    x = x.double().numpy().reshape(*x.shape[:-1], 8, 16)
    s = nearest_code(_finite_amax(x), np.full(x.shape[:-1], 6.0 * g), E4M3)
    unit = np.broadcast_to((E4M3[s] * g)[..., None], x.shape)
    nan = np.isnan(x).any(-1)
    ax = np.minimum(np.where(np.isnan(x), 0.0, np.abs(x)), 1e300)
    code = np.where(unit > 0, nearest_code(ax, np.where(unit > 0, unit, 1.0), E2M1), 0)
    code = code | (np.signbit(x).astype(np.int64) << 3)
    s = np.where(nan, 0x7F, s)
    return torch.from_numpy(code.reshape(*x.shape[:-2], 128).astype(np.uint8)), torch.from_numpy(s.astype(np.uint8))


class Record:
    """Byte places of a 4-bit cache's record, one value at a time, from the documented layout."""

    def __init__(self, bs):
        self.bs = bs

    def code(self, kind, slot, dim):
        byte = dim // 2
        if kind and slot & 2:
            byte ^= 32
        return 64 * self.bs * kind + 64 * slot + byte, 4 * (dim % 2)

    def scale(self, kind, slot, group):
        if not kind:
            return 128 * self.bs + 8 * slot + group
        t = slot % 16
        return 136 * self.bs + (slot // 16) * 128 + group * 16 + 4 * ((t & 3) ^ ((t >> 2) & 1)) + (t >> 2)

    def tables(self):
        """(code byte [2, bs, 128], shift [128], scale byte [2, bs, 8])."""
        c = torch.tensor([[[self.code(k, t, d)[0] for d in range(128)] for t in range(self.bs)] for k in range(2)])
        s = torch.tensor([[[self.scale(k, t, b) for b in range(8)] for t in range(self.bs)] for k in range(2)])
        return c, torch.arange(128) % 2 * 4, s


def write4(cache: torch.Tensor, bs, kind, slots, heads_codes, heads_scales):
    """Rows codes [T, Hk, 128], scales [T, Hk, 8] into the CPU cache [NB, Hk, 144 bs] at slots (negative: none)."""
    c, shift, s = Record(bs).tables()
    for t, slot in enumerate(slots.tolist()):
        if slot < 0 or slot >= cache.shape[0] * bs:
            continue
        rec = cache[slot // bs]
        o = slot % bs
        even, odd = heads_codes[t][:, 0::2], heads_codes[t][:, 1::2]
        rec[:, c[kind, o, 0::2]] = even | (odd << 4)
        rec[:, s[kind, o]] = heads_scales[t]


def read4(cache: torch.Tensor, bs, kind, blocks, offsets, g):
    """(code * group scale, value) float64 [n, Hk, 128] of slots `offsets` of `blocks` in the CPU cache."""
    c, shift, s = Record(bs).tables()
    blocks, offsets = torch.as_tensor(blocks), torch.as_tensor(offsets)
    rec = cache[blocks]                                             # [n, Hk, bytes]
    at = c[kind, offsets][:, None].expand(-1, cache.shape[1], -1)
    code = (rec.gather(2, at) >> shift.to(torch.uint8)) & 15
    table = torch.from_numpy(np.concatenate([E2M1, -E2M1]))
    scale = rec.gather(2, s[kind, offsets][:, None].expand(-1, cache.shape[1], -1))
    scale = scale.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    x = table[code.long()] * scale
    return x, x * float(np.float32(g))


def random_cache4(NB, Hk, bs, g, generator, wild=False):
    """A CPU cache of quantised normals (wild: random codes and scales over the whole range instead)."""
    if wild:
        cache = torch.randint(0, 256, (NB, Hk, 144 * bs), generator=generator, dtype=torch.uint8)
        scales = cache[..., 128 * bs:]
        scales.copy_(torch.where((scales & 0x7F) == 0x7F, scales & 0xFE, scales) & 0x7F)
        return cache
    cache = torch.zeros(NB, Hk, 144 * bs, dtype=torch.uint8)
    slots = torch.arange(NB * bs)
    for kind in range(2):
        x = torch.randn(NB * bs, Hk, 128, generator=generator).to(torch.bfloat16)
        codes, scales = quantize_rows4(x, g)
        write4(cache, bs, kind, slots, codes, scales)
    return cache


def decode64(q, cache, tables, lens, bs, scale, ks, vs, window=0, sinks=None):
    """(out float64 [S, H, 128], tolerance of a bf16 result, likewise).

    Tolerance, per element, with w the weights, W = sum w |v|, A_t = scale sum_d |q_d k_td|:
      2^-11 W               P in one f16 (half a step)
      2^-25 n max|v|        P below f16's normal range (the largest weight is at least 1 in its units)
      2 max_t A_t 2^-16 W   logits: 128 products summed in binary32 (2^-23 each at most), in numerator and sum
      n 2^-22 W             sums over the tokens in binary32, ex2 (2^-22)
      2^-8 |o|              the output's rounding, and bf16's smallest step
    """
    S, H, _ = q.shape
    Hk = cache.shape[1]
    out = torch.zeros(S, H, 128, dtype=torch.float64)
    tol = torch.zeros_like(out)
    cap = tables.shape[1] * bs
    for i in range(S):
        n = min(max(int(lens[i]), 0), cap)
        lo = max(0, n - window) if window else 0
        if n <= lo:
            continue
        pos = torch.arange(lo, n)
        ids = tables[i, pos // bs].long()
        k = read4(cache, bs, 0, ids, pos % bs, ks)[1]
        v = read4(cache, bs, 1, ids, pos % bs, vs)[1]
        for h in range(H):
            key, val = k[:, h // (H // Hk)], v[:, h // (H // Hk)]
            qq = q[i, h].double()
            z = key @ qq * scale
            a = (key.abs() @ qq.abs() * abs(scale)).max()
            top = z.max() if sinks is None else torch.maximum(z.max(), sinks[h].double())
            w = (z - top).exp()
            total = w.sum() + (0 if sinks is None else (sinks[h].double() - top).exp())
            w = w / total
            out[i, h] = w @ val
            W = w @ val.abs()
            m = n - lo
            own = w.max() if sinks is not None else 1.0             # a sink's share leaves less to the tokens
            tol[i, h] = ((2.0 ** -11 + 2 * a * 2.0 ** -16 + m * 2.0 ** -22) * W + 2.0 ** -25 * m * val.abs().max() * min(1.0, float(own) * m)
                         + out[i, h].abs() * 2.0 ** -8 + 2.0 ** -133)
    return out, tol
