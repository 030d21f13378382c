"""Decode attention over the 4-bit cache against the plain form in 64 bits (tolerances: lowbits_util.decode64)."""

import pathlib
import subprocess
import sys
import threading

import pytest
import torch

import paged_kv_decode_pda_gb300 as pda
from tests import lowbits_util as U

pytestmark = pytest.mark.gpu
DEV = "cuda"
KS, VS = 0.0043, 0.0039


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Batch:
    """A call's inputs on the CPU: shuffled pages; what no token fills holds NaN scales, unused entries a foreign block."""

    def __init__(self, lens, H, Hk, bs, seed=0, extra=1, q_scale=1.0, wild=False):
        g = gen(seed)
        self.lens, self.bs, self.H, self.Hk = list(lens), bs, H, Hk
        need = [-(-n // bs) for n in lens]
        NB = sum(need) + 2
        perm = torch.randperm(NB, generator=g).tolist()
        self.tables = torch.full((len(lens), max(need + [1]) + extra), perm[-1], dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.tables[i, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
            at += n
        self.cache = U.random_cache4(NB, Hk, bs, KS, g, wild=wild)
        used = torch.zeros(NB, bs, dtype=torch.bool)
        for i, n in enumerate(lens):
            p = torch.arange(n)
            used[self.tables[i, p // bs].long(), p % bs] = True
        _, _, s = U.Record(bs).tables()
        for b, o in torch.nonzero(~used).tolist():
            for kind in range(2):
                self.cache[b][:, s[kind, o]] = 0x7F
        self.q = (torch.randn(len(lens), H, 128, generator=g) * q_scale).to(torch.bfloat16)
        self.scale = 128 ** -0.5

    def run(self, **kw):
        lens = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        if kw.get("sinks") is not None:
            kw["sinks"] = kw["sinks"].to(DEV)
        return pda.decode_fp4(self.q.to(DEV), self.cache.to(DEV), self.tables.to(DEV), lens, self.scale, KS, VS, **kw)

    def check(self, got=None, scale=None, **kw):
        if got is None:
            got = self.run(**kw)
        want, tol = U.decode64(self.q, self.cache, self.tables, self.lens, self.bs, self.scale, KS, VS, **kw)
        err = (got.double().cpu() - want).abs()
        assert torch.isfinite(got.float()).all()
        assert (err <= tol).all(), (float(err.max()), float((err / tol).max()), torch.nonzero(err > tol)[:4].tolist())
        assert pda.query_device_status() == 0


@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 1), (8, 1), (32, 8), (40, 8), (6, 2), (21, 3)])
@pytest.mark.parametrize("bs", [16, 32, 48, 64, 80, 96, 112, 128])
def test_shapes(H, Hk, bs):
    Batch([1, 15, 16, 17, 100, 0, 129, 300], H, Hk, bs, seed=H + bs).check()


@pytest.mark.parametrize("lens", [[0], [1], [0, 0, 0], [128], [127, 1, 0, 0, 257], [1000], list(range(40)), [5] * 70 + [900]])
def test_lengths(lens):
    Batch(lens, 8, 2, 16, seed=len(lens)).check()


@pytest.mark.parametrize("window", [1, 7, 16, 100, 128, 1000, 1 << 30])
@pytest.mark.parametrize("bs", [16, 48, 128])
def test_window(window, bs):
    Batch([1, 16, 33, 250, 0, 400], 10, 2, bs, seed=window % 97).check(window=window)


@pytest.mark.parametrize("window", [0, 20])
def test_sinks(window):
    b = Batch([0, 1, 40, 300], 16, 4, 32, seed=3)
    sinks = torch.randn(16, generator=gen(5)) * 4
    sinks[3], sinks[7] = 30.0, -40.0
    b.check(sinks=sinks, window=window)


def test_e4m3_output():
    b = Batch([3, 77, 200], 8, 2, 16, seed=8)
    got = b.run(output_scale=0.01).cpu()
    assert got.dtype == torch.float8_e4m3fn
    want, tol = U.decode64(b.q, b.cache, b.tables, b.lens, 16, b.scale, KS, VS)
    want = want / 0.01
    # what the kernel rounds is off by the tolerance less bf16's step; then half an e4m3 step (2^-4, 2^-10 below its normals)
    far = tol / 0.01
    limit = far + (want.abs() + far) * 2.0 ** -4 + 2.0 ** -10
    assert ((got.double() - want.clamp(-448, 448)).abs() <= limit).all()
    assert pda.query_device_status() == 0


def test_large_queries():
    """Rows of far apart magnitudes; a negative scale."""
    b = Batch([50, 200], 8, 2, 16, seed=11)
    b.q = b.q * torch.tensor([1e-30, 1.0, 1e30, 0.0, 1e4, 1e-4, 3.0, 1e38]).view(1, 8, 1).to(torch.bfloat16)
    b.q[:, [2, 7]] = b.q[:, [2, 7]] * 0.0
    b.scale = -b.scale / 1e3
    b.check()


@pytest.mark.parametrize("size", [0, 20, 24, 27, 28, 30, 40, 80, 110])
@pytest.mark.parametrize("lens,bs", [([20, 5], 16), ([300], 128), ([5000], 16)])
def test_far_logits(size, lens, bs):
    """Logits of 2^size: where the largest is far in front its value comes out; a page named twice is weighted as once."""
    b = Batch(lens, 8, 2, bs, seed=60)
    b.tables[0, 1] = b.tables[0, 0] if lens[0] >= 2 * bs else b.tables[0, 1]
    far = 0
    for spread in (1.0, 2.0 ** size):
        b.q = (torch.randn(len(lens), 8, 128, generator=gen(61)) * spread).to(torch.bfloat16)
        b.scale = 2.0 ** size / spread if size < 40 else 128 ** -0.5
        got = b.run().double().cpu()
        assert torch.isfinite(got).all()
        for i, n in enumerate(lens):
            pos = torch.arange(n)
            ids = b.tables[i, pos // bs].long()
            k, v = (U.read4(b.cache, bs, kind, ids, pos % bs, s)[1] for kind, s in ((0, KS), (1, VS)))
            for h in range(8):
                z = k[:, h // 4] @ b.q[i, h].double() * b.scale
                a = (k[:, h // 4].abs() @ b.q[i, h].double().abs()).max() * b.scale
                top = z == z.max()
                rest = z[~top].max()
                if float(z.max() - rest) < 40 + float(a) * 2.0 ** -15:     # the rest: 2^-57 at most, wherever 128 sums in binary32 put it
                    continue
                far += 1
                want = v[top, h // 4].mean(0)
                # equal logits have equal weights; P, the output and the sums of few terms round
                assert ((got[i, h] - want).abs() <= v[top, h // 4].abs().mean(0) * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -16)).all(), (i, h)
    assert far >= (0 if size <= 20 else 8)
    assert pda.query_device_status() == 0


def test_wild_codes():
    """Codes and group scales over their whole range: exact products, logits far apart."""
    b = Batch([64, 130], 4, 2, 16, seed=12, wild=True, q_scale=0.02)
    b.check()


@pytest.mark.parametrize("lens,H,Hk,bs", [([9000], 4, 1, 16), ([70000], 8, 1, 64), ([70000, 3], 2, 2, 128), ([20000, 50, 0, 6000, 1], 5, 1, 32)])
def test_long(lens, H, Hk, bs):
    """One unit over many CTAs: pieces, and pieces joined in groups."""
    b = Batch([64 * 2], H, Hk, bs, seed=1)
    g = gen(2)
    # one small pool whose blocks the long rows name again and again
    NB = b.cache.shape[0] - 2
    b.cache = U.random_cache4(NB + 2, Hk, bs, KS, g)
    b.lens = lens
    b.tables = torch.randint(0, NB + 2, (len(lens), max(-(-n // bs) for n in lens) + 1), generator=g, dtype=torch.int32)
    b.q = torch.randn(len(lens), H, 128, generator=g).to(torch.bfloat16) * 3
    b.check()
    first = b.run()
    for _ in range(5):
        assert torch.equal(first, b.run())                     # which CTA joins the pieces changes nothing


def test_many_sequences():
    g = gen(21)
    lens = torch.randint(0, 40, (1500,), generator=g).tolist()
    lens[700] = 3000
    Batch(lens, 4, 1, 16, seed=22).check()


@pytest.mark.parametrize("H,Hk,bs", [(32, 8, 16), (40, 8, 64), (4, 4, 48), (8, 2, 16), (6, 2, 32), (8, 1, 128), (21, 3, 16), (16, 4, 128)])
@pytest.mark.parametrize("window,with_sinks", [(0, False), (100, True), (333, False)])
def test_wide_tables(H, Hk, bs, window, with_sinks):
    """Tables with room for long contexts: the larger chunks, by every number of heads to a unit."""
    b = Batch([1, 63, 64, 65, 255, 256, 257, 0, 1100, 16, 513, 500], H, Hk, bs, seed=H + bs + window, extra=8000)
    b.check(window=window, sinks=torch.randn(H, generator=gen(6)) if with_sinks else None)


def test_lengths_below_zero_are_empty():
    b = Batch([40, 0, 64], 4, 2, 16, seed=2)
    want = b.run()
    b.lens = [40, -5, 64]
    assert torch.equal(want, b.run())
    b.lens = [40, -(1 << 31), 64]
    assert torch.equal(want, b.run())


def test_threads_on_one_stream():
    """Calls of several threads on one stream take the workspace one after the other."""
    batches = [Batch([500, 30, 2000], 8, 2, 16, seed=61), Batch([100, 900], 40, 8, 32, seed=62), Batch([1, 7000], 8, 1, 64, seed=63)]
    want = [b.run() for b in batches]
    dev = [[x.to(DEV) for x in (b.q, b.cache, b.tables, torch.tensor(b.lens, dtype=torch.int32))] for b in batches]
    torch.cuda.synchronize()
    outs = [[] for _ in batches]

    def work(i):
        with torch.cuda.stream(stream):
            for _ in range(30):
                outs[i].append(pda.decode_fp4(*dev[i], 128 ** -0.5, KS, VS))

    stream = torch.cuda.Stream()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(batches))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(len(batches)):
        assert len(outs[i]) == 30 and all(torch.equal(x, want[i]) for x in outs[i])
    assert pda.query_device_status() == 0


def test_first_call_of_a_process_is_captured():
    """reserve_fp4, then a capture: nothing of the kernels was loaded before."""
    code = """
import torch, paged_kv_decode_pda_gb300 as pda
from tests.test_gpu_decode_fp4 import Batch, DEV, KS, VS
b = Batch([500, 30, 2000], 8, 2, 16, seed=31)
d = [x.to(DEV) for x in (b.q, b.cache, b.tables, torch.tensor(b.lens, dtype=torch.int32))]
out = torch.zeros_like(d[0])
side = torch.cuda.Stream()
pda.reserve_fp4(side)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=side):
    pda.decode_fp4(*d, 128 ** -0.5, KS, VS, out=out)
graph.replay()
torch.cuda.synchronize()
b.check(got=out)
"""
    root = pathlib.Path(__file__).resolve().parent.parent
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_released_and_made_again():
    b = Batch([500, 30, 2000], 8, 2, 16, seed=31)
    want = b.run()
    torch.cuda.synchronize()
    pda.release()
    assert torch.equal(want, b.run())


def test_lengths_past_the_table_row_are_cut():
    b = Batch([40, 64], 4, 2, 16, seed=2, extra=0)
    want = b.run()
    b.lens = [40, 1000]
    assert torch.equal(want, b.run())


def test_bad_block_is_flagged():
    b = Batch([40, 20], 4, 2, 16, seed=2)
    good = b.run()
    b.tables[0, 1] = 1 << 20
    got = b.run()
    assert pda.query_device_status() == 64
    assert torch.equal(got[1], good[1])
    b.tables[0, 1] = -1
    b.run()
    assert pda.query_device_status() == 64


def test_far_records():
    """Records past 2^32 bytes."""
    Hk, bs = 8, 64
    NB = (1 << 32) // (Hk * 144 * bs) + 40
    small = Batch([300], 32, Hk, bs, seed=4)
    cache = torch.empty(pda.fp4_cache_shape(NB, Hk, bs), dtype=torch.uint8, device=DEV)
    n = small.cache.shape[0]
    cache[NB - n:] = small.cache.to(DEV)
    got = pda.decode_fp4(small.q.to(DEV), cache, (small.tables + NB - n).to(DEV),
                         torch.tensor(small.lens, dtype=torch.int32, device=DEV), small.scale, KS, VS)
    small.check(got=got)


def test_streams_and_graphs():
    """Calls on two streams at once, and a graph replayed on other lengths; a capture without a workspace is refused."""
    a, b = Batch([500, 30, 2000], 8, 2, 16, seed=31), Batch([100, 900], 40, 8, 32, seed=32)
    want = [a.run(), b.run()]
    a_dev = [x.to(DEV) for x in (a.q, a.cache, a.tables, torch.tensor(a.lens, dtype=torch.int32))]
    b_dev = [x.to(DEV) for x in (b.q, b.cache, b.tables, torch.tensor(b.lens, dtype=torch.int32))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(20):
        for i, d in enumerate((a_dev, b_dev)):
            with torch.cuda.stream(streams[i]):
                outs[i].append(pda.decode_fp4(*d, 128 ** -0.5, KS, VS))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in outs[i])

    side = torch.cuda.Stream()
    out = torch.zeros_like(a_dev[0])
    graph = torch.cuda.CUDAGraph()
    refused = None
    with torch.cuda.graph(graph, stream=side):
        out.zero_()
        try:
            pda.decode_fp4(*a_dev, 128 ** -0.5, KS, VS, out=out)
        except pda.PdaError as e:
            refused = e.status
    assert refused == pda.PDA_ERR_WORKSPACE
    pda.reserve_fp4(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pda.decode_fp4(*a_dev, 128 ** -0.5, KS, VS, out=out)
    for lens in ([500, 30, 2000], [1, 0, 64], [400, 1, 1999], [500, 30, 2000]):
        a_dev[3].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        a.lens = lens
        a.check(got=out)
    assert torch.equal(out, want[0])


def test_serving_steps():
    """Steps as a server takes them: pages grow and fork on the device, tokens are rotated and written in 4 bits, and attended to."""
    bs, Hk, H, NB, R = 16, 2, 8, 40, 4
    g = gen(40)
    cache = torch.zeros(pda.fp4_cache_shape(NB, Hk, bs), dtype=torch.uint8, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    refs, tables, lens = torch.zeros(NB, **i32), torch.zeros(R, 6, **i32), torch.zeros(R, **i32)
    freq, mag = pda.rope_frequencies(128)

    def step(rows, add):
        pda.grow_pages(refs, tables, lens, torch.tensor(rows, **i32), torch.tensor([add] * len(rows), **i32), bs)
        L = lens.cpu()
        pos = torch.cat([torch.arange(int(L[r]) - add, int(L[r])) for r in rows])
        row = torch.tensor([r for r in rows for _ in range(add)])
        slots = tables.cpu()[row, pos // bs].long() * bs + pos % bs
        q = torch.randn(len(rows) * add, H, 128, generator=g).to(torch.bfloat16).to(DEV)
        k, v = (torch.randn(len(rows) * add, Hk, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
        q, k = pda.rope(q, k, pos.to(DEV), freq, magnitude=mag)
        pda.reshape_and_cache_fp4(k, v, cache, slots.to(DEV), KS, VS)
        return q

    step([0, 1], 37)                                            # two prompts
    pda.fork_pages(refs, tables, lens, torch.tensor([0, 0], **i32), torch.tensor([2, 3], **i32), bs, [cache])
    for _ in range(12):
        q = step([0, 1, 2, 3], 1)
        out = pda.decode_fp4(q, cache, tables, lens, 128 ** -0.5, KS, VS)
        want, tol = U.decode64(q.cpu(), cache.cpu(), tables.cpu(), lens.tolist(), bs, 128 ** -0.5, KS, VS)
        assert ((out.double().cpu() - want).abs() <= tol).all()
    pda.free_pages(refs, tables, lens, torch.tensor([0], **i32), bs)
    pda.compact_pages(refs, tables, lens, bs, [cache])
    q = step([1, 2, 3], 2)[1::2].contiguous()
    out = pda.decode_fp4(q, cache, tables[1:], lens[1:], 128 ** -0.5, KS, VS)
    want, tol = U.decode64(q.cpu(), cache.cpu(), tables.cpu()[1:], lens.tolist()[1:], bs, 128 ** -0.5, KS, VS)
    assert ((out.double().cpu() - want).abs() <= tol).all()
    # the cache read back is what was attended to
    starts = torch.cat([torch.zeros(1, dtype=torch.int32), lens.cpu().cumsum(0).to(torch.int32)]).to(DEV)
    k, v = pda.gather_cache_fp4(cache, tables, starts, int(starts[-1]), KS, VS)
    pos = torch.cat([torch.arange(n) for n in lens.tolist()])
    row = torch.repeat_interleave(torch.arange(R), lens.cpu().long())
    b = tables.cpu()[row, pos // bs].long()
    for got, kind, s in ((k, 0, KS), (v, 1, VS)):
        x = U.read4(cache.cpu(), bs, kind, b, pos % bs, 1.0)[0]
        assert torch.equal(got.cpu(), (x.float() * torch.tensor(s)).to(torch.bfloat16))
    assert pda.query_device_status() == 0


def test_slot_scale_steps():
    """Rows written with their own scales, attended to by decode_slot_scales and read back in the same values."""
    bs, Hk, H, NB = 16, 2, 8, 12
    g = gen(41)
    lens = [70, 33, 1]
    need = [-(-n // bs) for n in lens]
    perm = torch.randperm(NB, generator=g).to(torch.int32)
    tables = torch.zeros(3, 5, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
    pos = torch.cat([torch.arange(n) for n in lens])
    row = torch.repeat_interleave(torch.arange(3), torch.tensor(lens))
    slots = tables[row, pos // bs].long() * bs + pos % bs
    loud = torch.randn(len(pos), 1, 1, generator=g).exp()
    k, v = ((torch.randn(len(pos), Hk, 128, generator=g) * loud).to(torch.bfloat16).to(DEV) for _ in range(2))
    kc = torch.full((NB, Hk, 8, bs, 16), 0x7F, dtype=torch.uint8, device=DEV)
    vc = torch.full((NB, Hk, 128, bs), 0x7F, dtype=torch.uint8, device=DEV)
    ks, vs = (torch.full((NB, Hk, bs), float("nan"), device=DEV) for _ in range(2))
    pda.reshape_and_cache_slot_scales(k, v, kc, vc, ks, vs, slots.to(DEV))
    q = torch.randn(3, H, 128, generator=g).to(torch.bfloat16)
    lens_dev = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = pda.decode_slot_scales(q.to(DEV), kc, vc, ks, vs, tables.to(DEV), lens_dev, 128 ** -0.5).double().cpu()
    starts = torch.tensor([0, 70, 103, 104], dtype=torch.int32, device=DEV)
    gk, gv = pda.gather_cache_slot_scales(kc, vc, ks, vs, tables.to(DEV), starts, 104)
    codes, scales = U.quantize_rows8(k.cpu(), 2.0 ** -20)
    key = codes.view(torch.float8_e4m3fn).double() * scales.double()[..., None]
    codes, scales = U.quantize_rows8(v.cpu(), 2.0 ** -20)
    val = codes.view(torch.float8_e4m3fn).double() * scales.double()[..., None]
    # half a bf16 step, and the product's binary32 step before it
    assert ((gk.double().cpu() - key).abs() <= key.abs() * (2.0 ** -8 + 2.0 ** -22)).all()
    assert ((gv.double().cpu() - val).abs() <= val.abs() * (2.0 ** -8 + 2.0 ** -22)).all()
    for i in range(3):
        a, b = int(starts[i]), int(starts[i + 1])
        for h in range(H):
            w = torch.softmax(key[a:b, h // 4] @ q[i, h].double() * 128 ** -0.5, 0)
            want = w @ val[a:b, h // 4]
            W = w @ val[a:b, h // 4].abs()
            size = (key[a:b, h // 4].abs() @ q[i, h].double().abs()).max() * 128 ** -0.5
            assert ((out[i, h] - want).abs() <= want.abs() * 2.0 ** -8 + W * (2.0 ** -20 + 2 * size * 2.0 ** -16 + 100 * 2.0 ** -22)).all()
    assert pda.query_device_status() == 0
