"""The operators as a serving loop uses them: grow, rotate and write, attend to the chunk, fork, decode, free, compact."""

import torch
import pytest

import paged_kv_decode_pda_gb300 as pda
from tests import ops_util as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_chunked_prompts_forked_decoded_and_compacted():
    H, Hk, bs, NB, rows, cols = 8, 2, 16, 96, 6, 24
    g = torch.Generator().manual_seed(0)
    i32 = torch.int32
    refs = torch.zeros(NB, dtype=i32, device=DEV)
    tables = torch.zeros(rows, cols, dtype=i32, device=DEV)
    lens = torch.zeros(rows, dtype=i32, device=DEV)
    kc = torch.full((NB, Hk, 8, bs, 16), 0x7F, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    vc = torch.full((NB, Hk, 128, bs), 0x7F, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    f, mag = pda.rope_frequencies(128, scaling=pda.PDA_ROPE_RAMP, factor=4.0, original_length=64.0)
    ks, vs, scale = 0.05, 0.05, 128 ** -0.5
    keys = [torch.zeros(0, Hk, 128, dtype=torch.float64) for _ in range(rows)]
    vals = [torch.zeros(0, Hk, 128, dtype=torch.float64) for _ in range(rows)]

    def t32(x):
        return torch.tensor(x, dtype=i32, device=DEV)

    def step(which, new):
        """new[i] more tokens for row which[i], attended to; checked against the history in 64 bits."""
        before = lens.cpu().tolist()
        pda.grow_pages(refs, tables, lens, t32(which), t32(new), bs)
        T = sum(new)
        qkv = torch.randn(T, (H + 2 * Hk) * 128, generator=g).to(torch.bfloat16)
        pos = torch.cat([torch.arange(before[r], before[r] + n) for r, n in zip(which, new)])
        row = torch.cat([torch.full((n,), r) for r, n in zip(which, new)])
        tab = tables.cpu().long()
        slots = tab[row, pos // bs] * bs + pos % bs
        d = qkv.to(DEV)
        q, k, v = (x.view(T, -1, 128) for x in (d[:, :H * 128], d[:, H * 128:(H + Hk) * 128], d[:, (H + Hk) * 128:]))
        qr = pda.rope_and_cache(q, k, v, pos.to(DEV), slots.to(DEV), f, kc, vc, ks, vs, magnitude=mag)
        starts = t32([0] + torch.tensor(new).cumsum(0).tolist())
        rows_t = t32(which).long()
        out = pda.extend(qr, kc, vc, tables[rows_t].contiguous(), lens[rows_t].contiguous(), starts, scale, ks, vs)
        if all(n == 1 for n in new):
            dec = pda.decode(qr, kc, vc, tables[rows_t].contiguous(), lens[rows_t].contiguous(), scale, ks, vs)
        assert pda.query_device_status() == 0
        k64 = O.rope64(k.cpu(), pos, f, mag)
        # what the cache holds is e4m3; the rotated queries are bf16: the reference goes on from the bits themselves
        at = 0
        for r, n in zip(which, new):
            sl = slice(at, at + n)
            kq = kc.view(torch.uint8).cpu()[slots[sl] // bs, :, :, slots[sl] % bs].reshape(n, Hk, 128).view(O.FP8).double() * ks
            assert ((kq - k64[sl]).abs() <= 2.0 ** -4 * k64[sl].abs() + ks * 2.0 ** -10 + 1e-5).all()
            vq = (v[sl].cpu().float() / torch.tensor(vs)).clamp(-448, 448).to(torch.float8_e4m3fn).double() * vs
            keys[r], vals[r] = torch.cat([keys[r], kq]), torch.cat([vals[r], vq])
            K, V = keys[r].repeat_interleave(H // Hk, 1), vals[r].repeat_interleave(H // Hk, 1)
            L = K.shape[0]
            z = torch.einsum("nhd,thd->hnt", qr[sl].cpu().double(), K) * scale
            z = z.masked_fill(torch.arange(L)[None] > torch.arange(L - n, L)[:, None], float("-inf"))
            w = z.softmax(-1)
            ref, spread = torch.einsum("hnt,thd->nhd", w, V), torch.einsum("hnt,thd->nhd", w, V.abs())
            O.check_rows(out[sl], ref, spread, "extend")
            if all(m == 1 for m in new):
                O.check_rows(dec[sl], ref, spread, "decode")
            at += n

    step([0, 1], [50, 7])                 # prompts
    step([0, 1, 2], [33, 1, 100])         # a second chunk beside a decoding row and a new prompt
    pda.fork_pages(refs, tables, lens, t32([0, 2]), t32([3, 4]), bs, (kc, vc))
    for c, p in ((3, 0), (4, 2)):
        keys[c], vals[c] = keys[p].clone(), vals[p].clone()
    step([0, 1, 2, 3, 4], [1] * 5)        # branches part ways
    step([3, 4, 0], [1, 4, 1])
    pda.free_pages(refs, tables, lens, t32([0, 1]), bs)
    keys[0], vals[0], keys[1], vals[1] = keys[0][:0], vals[0][:0], keys[1][:0], vals[1][:0]
    pda.compact_pages(refs, tables, lens, bs, (kc, vc))
    live = int((refs > 0).sum())
    assert (refs[:live] > 0).all() and (refs[live:] == 0).all()
    step([2, 3, 4, 1], [1, 1, 1, 20])
    step([2, 3, 4], [1, 1, 1])
