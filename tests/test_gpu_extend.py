"""Attention of new tokens over the paged cache (pda_extend) against the 64-bit reference."""

import threading

import pytest
import torch

import paged_kv_decode_pda_gb300 as pda
from tests import ops_util as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def run(c, **kw):
    out = pda.extend(**c.to(DEV), **kw)
    assert pda.query_device_status() == 0
    return out


def check(c, label="", **kw):
    ref, spread = c.exact(window=kw.get("window", 0), sinks=kw.get("sinks"))
    dev = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in kw.items()}
    got = run(c, **dev)
    O.check_rows(got, ref, spread, label)
    return got, ref


@pytest.mark.parametrize("seqs", [
    [(1, 1)], [(1, 17)], [(2, 2)], [(16, 512)], [(5, 5), (1, 300), (0, 40), (0, 0), (33, 64)],
    [(130, 131), (64, 1000)], [(3, 129), (127, 127), (128, 128), (129, 129)], [(1, 128 * k + d) for k in (1, 2) for d in (-1, 0, 1)],
    [(300, 700), (1, 2000), (257, 257)]])
@pytest.mark.parametrize("H,Hk", [(4, 1), (8, 8), (16, 2)])
def test_lengths(seqs, H, Hk):
    check(O.Chunk(seqs, H, Hk, seed=len(seqs)))


@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 6, 7, 8])
def test_groups(g):
    check(O.Chunk([(45, 200), (7, 90), (1, 33)], 2 * g, 2, seed=g))


@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("bs", [16, 32, 48, 64, 80, 96, 112, 128])
def test_block_sizes_and_layouts(bs, shuffled):
    check(O.Chunk([(70, 333), (2, bs + 1), (9, 9), (140, 140)], 8, 2, bs, seed=bs, shuffled=shuffled))


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 128, 300, 5000])
def test_windows(window):
    check(O.Chunk([(200, 450), (1, 600), (4, 4), (130, 1000)], 8, 2, 32, seed=window), window=window)


@pytest.mark.parametrize("seqs", [[(1, 777)], [(90, 400), (1, 5)]])
@pytest.mark.parametrize("value", [-40.0, 0.0, 3.0, 60.0])
def test_sinks(seqs, value):
    sinks = torch.linspace(value - 2, value + 2, 8)
    check(O.Chunk(seqs, 8, 2, seed=1), sinks=sinks)


def test_more_rows_than_tokens_gives_zeros():
    c = O.Chunk([(6, 4), (5, 0), (200, 150), (1, 1)], 8, 2, seed=4)
    for sinks in (None, torch.zeros(8)):
        got, ref = check(c, sinks=sinks)
        for s, (n, L) in enumerate(c.seqs):
            none = max(0, n - L)
            assert (got[c.starts[s]:c.starts[s] + none] == 0).all()


def test_rows_of_no_sequence_stay_as_they_were():
    c = O.Chunk([(3, 70), (0, 8), (140, 150)], 8, 2, seed=6, pad_front=5, pad_back=131)
    mark = torch.full((c.T, 8, 128), -3.0, dtype=torch.bfloat16, device=DEV)
    run(c, out=mark)
    assert (mark[:5] == -3).all() and (mark[c.starts[-1]:] == -3).all()
    ref, spread = c.exact()
    O.check_rows(mark, ref, spread)


def test_e4m3_output():
    c = O.Chunk([(20, 300), (1, 64)], 8, 2, seed=8)
    ref, spread = c.exact()
    scale = 0.01
    got = run(c, output_scale=scale)
    assert got.dtype == torch.float8_e4m3fn
    want = (ref / scale).clamp(-448, 448)
    # half an e4m3 step (2^-4 relative, 2^-10 below the normal range) and the kernel's own error
    bound = torch.maximum(2.0 ** -4 * want.abs(), torch.tensor(2.0 ** -10, dtype=torch.float64)) + (1 + 2.0 ** -4) * O.WEIGHT_ERR * spread / scale
    assert ((got.cpu().double() - want).abs() <= bound).all()


@pytest.mark.parametrize("power", [-100, -20, 40, 100])
def test_query_rows_of_any_magnitude(power):
    c = O.Chunk([(40, 200), (1, 150)], 8, 2, seed=12)
    c.q = (c.q.float() * 2.0 ** power).to(torch.bfloat16)
    c.scale *= 2.0 ** -power
    check(c)


def test_a_dominant_token_leaves_room_for_the_rest():
    # one key far above all the others, many values of small weight behind it
    c = O.Chunk([(2, 1500)], 4, 1, seed=13)
    b = int(c.tables[0, 0])
    c.q = torch.full_like(c.q, 0.5)
    c.k_cache.view(torch.uint8)[b, :, :, 0, :] = torch.tensor(150.0).to(O.FP8).view(torch.uint8)
    check(c)


def test_pages_no_row_attends_to_are_not_read():
    # entries in front of the window name a block of NaN codes
    c = O.Chunk([(10, 1000)], 4, 1, seed=14)
    w = 60
    lo = max(0, 990 - w + 1) // c.bs
    ref, spread = c.exact(window=w)
    free = [b for b in range(c.NB) if b not in c.tables[0, :-(-1000 // c.bs)].tolist()][0]
    c.k_cache.view(torch.uint8)[free] = 0x7F
    c.v_cache.view(torch.uint8)[free] = 0xFF
    c.tables[0, :lo] = free
    O.check_rows(run(c, window=w), ref, spread)


def test_a_long_context_split_over_the_gpu():
    c = O.Chunk([(2, 20000)], 8, 1, seed=15)
    check(c)
    c = O.Chunk([(3, 9000), (1, 17)], 8, 2, seed=16)
    check(c)
    check(c, sinks=torch.linspace(-3, 6, 8))
    check(c, window=5000)


@pytest.mark.parametrize("seqs,H,Hk,bs", [
    ([(2, 700 + 150 * (i % 9)) for i in range(21)], 16, 8, 16),               # 168 items of few rows, the last 16 cut
    ([(70, 1100 + 37 * i) for i in range(20)] + [(1, 9), (0, 5)], 24, 8, 32),  # full tiles, and spare slots
    ([(9, 2000)] * 41, 32, 4, 64),
])
def test_more_items_than_sms(seqs, H, Hk, bs):
    c = O.Chunk(seqs, H, Hk, bs, seed=25)
    check(c)
    check(c, sinks=torch.linspace(-2, 4, H), window=900)


def test_a_cache_past_2_31_bytes():
    bs, Hk, NB = 16, 8, 140_000
    kc = torch.zeros(NB, Hk, 8, bs, 16, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    vc = torch.zeros(NB, Hk, 128, bs, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    assert kc.numel() > 1 << 31
    c = O.Chunk([(5, 100)], 16, Hk, bs, seed=17, garbage=False)
    n = -(-100 // bs)
    far = torch.arange(NB - n, NB)
    kc.view(torch.uint8)[far] = c.k_cache.view(torch.uint8)[c.tables[0, :n].long()].to(DEV)
    vc.view(torch.uint8)[far] = c.v_cache.view(torch.uint8)[c.tables[0, :n].long()].to(DEV)
    d = c.to(DEV)
    d.update(k_cache=kc, v_cache=vc)
    d["block_tables"][0, :n] = far.to(torch.int32)
    ref, spread = c.exact()
    O.check_rows(pda.extend(**d), ref, spread)


def test_single_tokens_agree_with_decode():
    c = O.Chunk([(1, n) for n in (1, 16, 100, 1000, 333)], 16, 2, seed=18)
    d = c.to(DEV)
    a = pda.extend(**d)
    b = pda.decode(d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["seq_lens"], c.scale, c.ks, c.vs)
    ref, spread = c.exact()
    O.check_rows(a, ref, spread)
    assert ((a.double() - b.double()).abs().cpu() <= 2.0 ** -7 * ref.abs() + 2 * O.WEIGHT_ERR * spread).all()


def test_the_same_call_gives_the_same_bits():
    c = O.Chunk([(200, 900), (1, 3000), (7, 50)], 8, 2, seed=19)
    d = c.to(DEV)
    a = pda.extend(**d)
    for _ in range(3):
        assert torch.equal(pda.extend(**d), a)


def test_the_same_bits_where_items_are_cut():
    # 40 x 8 items of one size: which of them the last round holds must not change
    c = O.Chunk([(3, 1500)] * 40, 16, 8, seed=26)
    d = c.to(DEV)
    a = pda.extend(**d)
    for _ in range(5):
        assert torch.equal(pda.extend(**d), a)


@pytest.mark.parametrize("scale,ks", [(-0.09, 0.05), (0.09, -0.05), (0.0, 0.05), (-0.09, -0.05)])
def test_scales_of_any_sign(scale, ks):
    c = O.Chunk([(40, 200), (1, 150)], 8, 2, seed=27)
    c.scale, c.ks = scale, ks
    check(c)
    check(c, window=(1 << 31) - 1)


def test_a_window_past_every_position_with_rows_in_front_of_the_cache():
    c = O.Chunk([(9, 4), (150, 120)], 8, 2, seed=28)
    check(c, window=(1 << 31) - 1)


@pytest.mark.parametrize("seqs", [[(40, 300), (1, 30)], [(2, 9000)], [(3, 400)] * 30])
def test_captured_without_a_workspace(seqs):
    c = O.Chunk(seqs, 8, 2 if len(seqs) < 9 else 8, seed=29)
    d = c.to(DEV)
    ref, spread = c.exact()
    s = torch.cuda.Stream(priority=-1)   # apart from the streams that other tests draw
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(d["q"])
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        pda.extend(**d, out=out)
    for _ in range(2):
        out.zero_()
        gr.replay()
    torch.cuda.synchronize()
    O.check_rows(out, ref, spread)


def test_two_batches_in_turn_on_one_stream():
    big, small = O.Chunk([(2, 9000), (2, 8000)], 8, 2, seed=20), O.Chunk([(3, 4000)], 8, 2, seed=21)
    outs = [(run(c), c) for c in (big, small, big)]
    for got, c in outs:
        ref, spread = c.exact()
        O.check_rows(got, ref, spread)


@pytest.mark.parametrize("seqs", [[(40, 100), (1, 30)], [(2, 9000)]])
def test_captured_and_on_another_stream(seqs):
    c = O.Chunk(seqs, 8, 2, seed=22)
    d = c.to(DEV)
    ref, spread = c.exact()
    s = torch.cuda.Stream(priority=-1)   # apart from the streams that other tests draw
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(d["q"])
    with torch.cuda.stream(s):
        pda.extend(**d, out=out)                       # sizes this stream's workspace
        gr = torch.cuda.CUDAGraph()
        s.synchronize()
        out.zero_()
        with torch.cuda.graph(gr, stream=s):
            pda.extend(**d, out=out)
        gr.replay()
        gr.replay()
    s.synchronize()
    O.check_rows(out, ref, spread)
    assert pda.query_device_status() == 0


def test_block_check_keeps_reads_in_the_pool():
    c = O.Chunk([(4, 100)], 4, 1, seed=23)
    c.tables[0, 1] = c.NB + 5
    pda.set_block_check(c.NB)
    try:
        d = c.to(DEV)
        pda.extend(**d)
        assert pda.query_device_status() == 64
    finally:
        pda.set_block_check(0)


def test_more_tiles_than_are_ordered():
    c = O.Chunk([(1, 1 + i % 5) for i in range(17000)], 1, 1, seed=31)
    check(c)


def test_threads_on_one_stream():
    # both batches have an order and cut items, which the workspace hands from kernel to kernel
    batches = [O.Chunk([(3, 1500 - 300 * i)] * 40, 16, 8, seed=32 + i).to(DEV) for i in range(2)]
    want = [pda.extend(**d) for d in batches]
    got = [[], []]

    def work(i):
        for _ in range(40):
            got[i].append(pda.extend(**batches[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 40 and all(torch.equal(x, want[i]) for x in got[i])


def test_nothing_to_do():
    c = O.Chunk([(0, 5), (0, 0)], 4, 1, seed=24, pad_back=3)
    mark = torch.full((c.T, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    run(c, out=mark)
    assert (mark == 7).all()


@pytest.mark.parametrize("lagging", [False, True])
@pytest.mark.parametrize("power", [12, 20, 24, 25, 26, 30, 60, 125])
@pytest.mark.parametrize("seqs,H,Hk", [
    ([(1, 1), (1, 5), (40, 300), (140, 400), (3, 2)], 8, 2), ([(2, 9000)], 8, 1), ([(3, 1500)] * 40, 16, 8)])
def test_logits_of_any_magnitude(seqs, H, Hk, power, lagging):
    # All tokens hold one value, so that the output is that value whatever the weights are. Lagging: the tokens' logits
    # go up by a small step (3.3 in log2 units at 2^25) from one tile of 128 tokens to the next.
    c = O.Chunk(seqs, H, Hk, seed=40, garbage=False)
    if lagging:
        c.q.zero_()
        c.q[..., 0] = 1 + torch.arange(c.T * H).view(c.T, H) % 128 / 128
        c.q[..., 127] = 2.0 ** -12
        kb = torch.zeros(c.NB, Hk, 8, 16, 16)
        kb[:, :, 0, :, 0] = 448
        for s, (_, n) in enumerate(seqs):
            for t in range(0, n, 16):
                kb[int(c.tables[s, t // 16]), :, 7, :, 15] = t // 128 % 16 * 0.25
        c.k_cache = kb.to(O.FP8)
        top = 448.0 * 2
    else:
        k = c.k_cache.double().permute(0, 3, 1, 2, 4).reshape(-1, Hk, 128)
        top = max((c.q[t].double().view(Hk, -1, 128) @ k.permute(1, 2, 0)).abs().max().item() for t in range(0, c.T, 7))
    c.scale = 2.0 ** power / (top * c.ks)
    v = torch.linspace(0.5, 2, Hk * 128).view(Hk, 128).to(O.FP8)
    c.v_cache = v[None, :, :, None].expand(c.NB, Hk, 128, 16).contiguous()
    want = (v.double() * c.vs).repeat_interleave(H // Hk, 0).expand(c.T, H, 128).clone()
    for s, (n, L) in enumerate(seqs):
        want[c.starts[s]:c.starts[s] + max(0, n - L)] = 0
    O.check_rows(run(c), want, want.abs())
    O.check_rows(run(c, sinks=torch.full((H,), -2e38, device=DEV)), want, want.abs())


@pytest.mark.parametrize("power", [4, 8, 12])
@pytest.mark.parametrize("seqs", [[(40, 300), (140, 400), (1, 5)], [(2, 9000)]])
def test_large_logits_against_64_bits(seqs, power):
    # logits below 2^power. With A the largest sum |q k| * scale, the fp32 sum of 128 products is off by at most
    # 128 * 2^-24 * A: relative, a weight's error and, once more, their sum's
    c = O.Chunk(seqs, 8, 2, seed=41)
    top = big = 0.0
    for s, (n, _) in enumerate(seqs):
        q = c.q[c.starts[s]:c.starts[s + 1]].double().view(n, 2, 4, 128).permute(1, 0, 2, 3).reshape(2, -1, 128)
        k = c.keys_values(s)[0].permute(1, 2, 0)
        top, big = max(top, (q @ k).abs().max().item()), max(big, (q.abs() @ k.abs()).max().item())
    c.scale = 2.0 ** power / top
    ref, spread = c.exact()
    # a weight below 2^-31 of the largest is below f16's smallest step once 2^7 stands for the largest (its half is
    # 2^-25, and the largest's place is off by less than one): it may vanish whole where all others meet zeros in V
    floor = max(n for _, n in seqs) * 2.0 ** -31 * 448 * c.vs
    O.check_rows(run(c), ref, spread * (1 + 2.0 ** -16 * big * c.scale / O.WEIGHT_ERR) + floor / O.WEIGHT_ERR)


@pytest.mark.parametrize("seqs,H,Hk", [
    ([(1 + 7 * i % 60, 1 + 7 * i % 60 + i % 50) for i in range(300)], 8, 8),                # one KV tile an item
    ([(1, 1 + i % 128) if i % 5 else (200 + i % 50, 120 + 40 * (i % 9)) for i in range(240)], 16, 2),
    ([(150, 40), (1, 100), (3, 5000), (128, 128)] * 30, 8, 4),                              # blocks without tiles
])
def test_items_of_few_tiles_in_a_row(seqs, H, Hk):
    # items that a block passes without a product, next to each other and next to long ones
    c = O.Chunk(seqs, H, Hk, seed=42)
    d = c.to(DEV)
    ref, spread = c.exact()
    a = pda.extend(**d, out=torch.zeros_like(d["q"]))
    O.check_rows(a, ref, spread)
    for _ in range(60):
        assert torch.equal(pda.extend(**d, out=torch.zeros_like(a)), a)
    assert pda.query_device_status() == 0


@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 200, 1 << 30, 9001])
def test_a_window_past_the_context_leaves_the_plan_as_it_is(window):
    # a call that splits the KV range: the same splits, and with them the same bits, as without a window
    c = O.Chunk([(2, 9000)], 8, 2, seed=43)
    d = c.to(DEV)
    assert torch.equal(pda.extend(**d, window=window), pda.extend(**d))


@pytest.mark.parametrize("reserved,seqs,H,Hk", [
    ((24, 12, 600), [(2, 9000)], 8, 8),                  # one split, no order
    ((4000, 500, 600), [(3, 4000), (1, 9)], 16, 2),      # an order
    ((4096, 1, 600), [(700, 3000)], 8, 1),               # splits, and more rows than the call's
    ((4000, 40, 100), [(3, 1500)] * 40, 16, 8),          # an order and pieces, fewer pages
])
def test_reserving_covers_smaller_calls(reserved, seqs, H, Hk):
    # captured on a stream whose workspace was sized for more: the plan, and so the bits, of the call outside a capture
    c = O.Chunk(seqs, H, Hk, seed=44)
    d = c.to(DEV)
    want = pda.extend(**d)
    T, S, MB = reserved
    assert T >= c.T and S >= len(seqs) and MB >= c.tables.shape[1]
    pda.release()
    s = torch.cuda.Stream(priority=-1)
    s.wait_stream(torch.cuda.current_stream())
    pda.reserve_extend(T, S, H, Hk, MB, c.bs, stream=s)
    s.synchronize()
    out = torch.zeros_like(d["q"])
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        pda.extend(**d, out=out)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("seqs,H,Hk", [
    ([(300, 700), (130, 131)], 8, 2),                # full tiles of both blocks
    ([(2, 9000), (1, 40)], 8, 2),                    # KV splits
    ([(3, 1500)] * 40, 16, 8),                       # cut pieces
    ([(70, 900 + 37 * i) for i in range(20)] + [(0, 5), (4, 2)], 24, 8)])
@pytest.mark.parametrize("sinks", [False, True])
def test_e4m3_output_on_every_path(seqs, H, Hk, sinks):
    c = O.Chunk(seqs, H, Hk, seed=45)
    s = torch.linspace(-2, 4, H) if sinks else None
    ref, spread = c.exact(sinks=s)
    scale = ref.abs().max().item() / 600                # some saturate
    got = run(c, output_scale=scale, sinks=None if s is None else s.to(DEV)).cpu().double()
    want = (ref / scale).clamp(-448, 448)
    # as in test_e4m3_output: half an e4m3 step, and the kernel's own error
    bound = torch.maximum(2.0 ** -4 * want.abs(), torch.tensor(2.0 ** -10, dtype=torch.float64)) \
        + (1 + 2.0 ** -4) * O.WEIGHT_ERR * spread / scale
    assert (want.abs() == 448).any() and ((got - want).abs() <= bound).all()


@pytest.mark.parametrize("rows,lens", [([3] * 24, [140_000 - 611 * i for i in range(24)]), ([2], [140_000]),
                                       ([40, 1], [135_000, 90])])
def test_contexts_past_the_sorted_sizes(rows, lens):
    # more than 1023 tiles of 128 tokens; against pda_decode, with each row as a sequence of its own
    H, Hk, bs = 16, 8, 64
    NB = -(-max(lens) // bs)
    g = torch.Generator(device=DEV).manual_seed(46)
    kc, vc = (torch.randint(0, 256, s, generator=g, dtype=torch.uint8, device=DEV).bitwise_and_(0xBF)   # below 2 in size
              for s in ((NB, Hk, 8, bs, 16), (NB, Hk, 128, bs)))
    tables = torch.stack([torch.randperm(NB, generator=g, device=DEV) for _ in rows]).to(torch.int32)
    q = torch.randn(sum(rows), H, 128, generator=g, device=DEV).to(torch.bfloat16)
    t32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    starts = t32([0] + torch.tensor(rows).cumsum(0).tolist())
    args = (128 ** -0.5, 0.8, 1.0)
    got = pda.extend(q, kc, vc, tables, t32(lens), starts, *args)
    of = torch.repeat_interleave(torch.arange(len(rows)), torch.tensor(rows))
    at = t32([n - m + 1 + i for n, m in zip(lens, rows) for i in range(m)])
    want, spread = (pda.decode(q, kc, v, tables[of.to(DEV)].contiguous(), at, *args).double()
                    for v in (vc, vc.bitwise_and(0x7F)))
    assert pda.query_device_status() == 0
    # half a bf16 step on either side, and the weights' error against a spread that is itself rounded to bf16
    assert ((got.double() - want).abs() <= 2.0 ** -7 * want.abs() + 2 * O.WEIGHT_ERR * spread * (1 + 2.0 ** -8)).all()
