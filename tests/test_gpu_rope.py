"""Rotary positions (pda_rope, pda_rope_and_cache) against 64-bit references."""

import pytest
import torch

import paged_kv_decode_pda_gb300 as pda
from tests import ops_util as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def inputs(T, H, Hk, seed, max_pos=5000):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, (H + 2 * Hk) * 128, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, max_pos, (T,), generator=g)
    return qkv, pos


def split(qkv, H, Hk):
    T = qkv.shape[0]
    return (qkv[:, :H * 128].view(T, H, 128), qkv[:, H * 128:(H + Hk) * 128].view(T, Hk, 128),
            qkv[:, (H + Hk) * 128:].view(T, Hk, 128))


def check_bf16(got, ref, x, n, mag, interleaved):
    """Half a bf16 step of the value (2^-8 relative); on rotated dims also the fp32 rotation: an angle off by at
    most 2e-7 rad (its 24-bit rounding, 2 pi 2^-26, and the sine's own error) and three roundings of 2^-24 on each
    product: below 5e-7 of |a| + |b|."""
    size = torch.zeros_like(ref)
    x = x.double()
    d0 = torch.arange(n) * 2 if interleaved else torch.arange(n)
    d1 = d0 + 1 if interleaved else d0 + n
    s = (x[..., d0].abs() + x[..., d1].abs()) * abs(mag)
    size[..., d0], size[..., d1] = s, s
    bound = 2.0 ** -8 * ref.abs() + 5e-7 * size
    err = (got.cpu().double() - ref).abs()
    assert (err <= bound).all(), (err - bound).max()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,Hk,rot", [
    (1, 1, 1, 128), (3, 8, 1, 64), (17, 40, 8, 128), (5, 7, 7, 96), (33, 4, 2, 32), (9, 3, 1, 20), (2, 2, 2, 2),
    (4, 4, 2, 0), (130, 32, 8, 128), (700, 12, 4, 16), (2501, 3, 1, 128)])
def test_rope(T, H, Hk, rot, interleaved):
    qkv, pos = inputs(T, H, Hk, seed=T + rot)
    q, k, _ = split(qkv, H, Hk)
    f = pda.rope_frequencies(rot)[0] if rot else torch.empty(0, dtype=torch.float64)
    qd, kd, _ = split(qkv.to(DEV), H, Hk)                       # strided views of the packed projection
    qo, ko = pda.rope(qd, kd, pos.to(DEV), f, magnitude=1.25, interleaved=interleaved)
    for got, x in ((qo, q), (ko, k)):
        assert got.is_contiguous()
        check_bf16(got, O.rope64(x, pos, f, 1.25, interleaved), x, rot // 2, 1.25, interleaved)
    # in place, on the views themselves
    pda.rope(qd, kd, pos.to(DEV), f, magnitude=1.25, interleaved=interleaved, q_out=qd, k_out=kd)
    assert torch.equal(qd, qo) and torch.equal(kd, ko)


@pytest.mark.parametrize("scaling", [pda.PDA_ROPE_LINEAR, pda.PDA_ROPE_BASE, pda.PDA_ROPE_RAMP, pda.PDA_ROPE_BANDS])
def test_scaled_frequencies_at_far_positions(scaling):
    f, mag = pda.rope_frequencies(128, scaling=scaling, factor=32.0, original_length=4096.0)
    qkv, _ = inputs(6, 2, 1, seed=3)
    pos = torch.tensor([0, 1, 131071, 999_983, -5, (1 << 24) + 1])
    q, k, _ = split(qkv, 2, 1)
    qd, kd, _ = split(qkv.to(DEV), 2, 1)
    qo, ko = pda.rope(qd, kd, pos.to(DEV), f, magnitude=mag)
    for got, x in ((qo, q), (ko, k)):
        check_bf16(got, O.rope64(x, pos, f, mag), x, 64, mag, False)


def test_a_turn_back_undoes_a_turn():
    q = torch.randn(4, 2, 128, device=DEV).to(torch.bfloat16)
    pos = torch.tensor([0, 17, 100000, 1 << 40], device=DEV)
    f, _ = pda.rope_frequencies(128)
    there, none = pda.rope(q, None, pos, f)
    back, _ = pda.rope(there, None, -pos, f)
    assert none is None and torch.equal(there[0], q[0])
    # two bf16 roundings, of values that rotate into each other
    size = q.float()[..., :64].abs() + q.float()[..., 64:].abs()
    assert ((back.float() - q.float()).abs() <= 2.0 ** -7 * size.repeat(1, 1, 2) * 1.01).all()


def test_views_off_the_16_byte_grid():
    T, H = 5, 3
    flat = torch.randn(T * (H * 130 + 7) + 1, device=DEV).to(torch.bfloat16)
    x = torch.as_strided(flat, (T, H, 128), (H * 130 + 7, 130, 1), 1)
    pos = torch.arange(T, device=DEV)
    f, _ = pda.rope_frequencies(128)
    got, _ = pda.rope(x, None, pos, f)
    check_bf16(got, O.rope64(x.cpu(), pos.cpu(), f), x.cpu(), 64, 1.0, False)


def to_code(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("T,H,Hk,bs,rot,interleaved,runs", [
    (1, 4, 1, 16, 128, False, False), (7, 8, 8, 32, 64, True, False), (64, 5, 1, 48, 128, False, True),
    (19, 6, 2, 128, 20, False, False), (300, 16, 2, 64, 128, True, False), (2500, 8, 8, 16, 96, False, True)])
def test_rope_and_cache(T, H, Hk, bs, rot, interleaved, runs, shuffled):
    qkv, pos = inputs(T, H, Hk, seed=T)
    g = torch.Generator().manual_seed(T + 1)
    NB = -(-T // bs) + 3
    if runs:
        slots = (torch.randperm(NB, generator=g)[torch.arange(T) // bs]) * bs + torch.arange(T) % bs
        slots[5:7] = -1
    else:
        slots = torch.randperm(NB * bs, generator=g)[:T]
        slots[::5] = -1
    ks, vs, mag = 0.05, 0.03, 1.1
    f = pda.rope_frequencies(rot)[0]
    kc = torch.randint(0, 256, (NB, Hk, 8, bs, 16), generator=g, dtype=torch.uint8)
    vc = torch.randint(0, 256, (NB, Hk, bs // 16, 128, 16) if shuffled else (NB, Hk, 128, bs), generator=g,
                       dtype=torch.uint8)
    q, k, v = split(qkv, H, Hk)
    qd, kd, vd = split(qkv.to(DEV), H, Hk)
    kcd, vcd = kc.to(DEV), vc.to(DEV)
    qo = pda.rope_and_cache(qd, kd, vd, pos.to(DEV), slots.to(DEV), f, kcd, vcd, ks, vs, magnitude=mag,
                            interleaved=interleaved, v_shuffled=shuffled)
    assert pda.query_device_status() == 0
    check_bf16(qo, O.rope64(q, pos, f, mag, interleaved), q, rot // 2, mag, interleaved)
    # the queries are the same, bit for bit, as without the cache
    assert torch.equal(qo, pda.rope(qd, None, pos.to(DEV), f, magnitude=mag, interleaved=interleaved)[0])
    # V: the codes of the binary32 quotient, exactly; K: e4m3 of the rotated key, where the value in 64 bits may lie
    # a rotation's error from a rounding border: half an e4m3 step (2^-4 relative, 2^-10 below 2^-6) and that error
    k64 = O.rope64(k, pos, f, mag, interleaved) / ks
    size = (k.double().abs().amax(-1, keepdim=True) * 2 * mag / ks).expand_as(k64)
    kg, vg = kcd.cpu(), vcd.cpu()
    kmask, vmask = torch.ones_like(kc, dtype=torch.bool), torch.ones_like(vc, dtype=torch.bool)
    vcode = to_code((v.float() / torch.tensor(vs, dtype=torch.float32)).clamp(-448, 448))
    for t, s in enumerate(slots.tolist()):
        if s < 0:
            continue
        b, o = divmod(s, bs)
        got = kg[b, :, :, o].reshape(Hk, 128).view(torch.float8_e4m3fn).double()
        want = k64[t].clamp(-448, 448)
        half = torch.maximum(2.0 ** -4 * want.abs(), torch.tensor(2.0 ** -10, dtype=torch.float64))
        assert ((got - want).abs() <= half + 1e-6 * size[t]).all()
        kmask[b, :, :, o] = False
        if shuffled:
            assert torch.equal(vg[b, :, o // 16, :, o % 16], vcode[t])
            vmask[b, :, o // 16, :, o % 16] = False
        else:
            assert torch.equal(vg[b, :, :, o], vcode[t])
            vmask[b, :, :, o] = False
    # everything else is as it was
    assert torch.equal(kg[kmask], kc[kmask]) and torch.equal(vg[vmask], vc[vmask])


@pytest.mark.parametrize("T", [3, 700])
@pytest.mark.parametrize("rot", [128, 20])
def test_a_slot_past_the_pool_is_skipped_and_flagged(T, rot):
    qkv, pos = inputs(T, 2, 2, seed=9)
    q, k, v = split(qkv.to(DEV), 2, 2)
    NB, bs = 50, 16
    slots = torch.arange(T)
    slots[1] = NB * bs
    kc, vc = torch.zeros(NB, 2, 8, bs, 16, dtype=torch.uint8, device=DEV), torch.zeros(NB, 2, 128, bs, dtype=torch.uint8, device=DEV)
    f = pda.rope_frequencies(rot)[0]
    pda.rope_and_cache(q, k, v, pos.to(DEV), slots.to(DEV), f, kc, vc, 0.05, 0.05)
    assert pda.query_device_status() == 16
    slots[1] = -1
    kr, vr = torch.zeros_like(kc), torch.zeros_like(vc)
    pda.rope_and_cache(q, k, v, pos.to(DEV), slots.to(DEV), f, kr, vr, 0.05, 0.05)
    assert pda.query_device_status() == 0 and torch.equal(kc, kr) and torch.equal(vc, vr)


def test_identity_rotation_writes_what_the_cache_writer_writes():
    T, Hk, bs, NB = 90, 4, 32, 8
    qkv, pos = inputs(T, 4, Hk, seed=2)
    q, k, v = split(qkv.to(DEV), 4, Hk)
    slots = torch.randperm(NB * bs)[:T].to(DEV)
    f = torch.zeros(64, dtype=torch.float64)
    a = [torch.zeros(NB, Hk, 8, bs, 16, dtype=torch.uint8, device=DEV), torch.zeros(NB, Hk, 128, bs, dtype=torch.uint8, device=DEV)]
    b = [x.clone() for x in a]
    qo = pda.rope_and_cache(q, k, v, pos.to(DEV), slots, f, *a, 0.05, 0.04)
    pda.reshape_and_cache(k.contiguous(), v.contiguous(), *b, slots, 0.05, 0.04)
    assert torch.equal(qo, q) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_and_on_another_stream():
    qkv, pos = inputs(40, 8, 2, seed=5)
    q, k, _ = split(qkv.to(DEV), 8, 2)
    f, _ = pda.rope_frequencies(128)
    pos = pos.to(DEV)
    want = pda.rope(q, k, pos, f)
    s = torch.cuda.Stream(priority=-1)   # apart from the streams that other tests draw
    s.wait_stream(torch.cuda.current_stream())
    qo, ko = torch.empty_like(want[0]), torch.empty_like(want[1])
    pda.rope(q, k, pos, f, q_out=qo, k_out=ko, stream=s)
    s.synchronize()
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        pda.rope(q, k, pos, f, q_out=qo, k_out=ko)
    pos.add_(1)
    gr.replay()
    again = pda.rope(q, k, pos, f)
    assert torch.equal(qo, again[0]) and torch.equal(ko, again[1])


def test_empty_and_misplaced():
    f, _ = pda.rope_frequencies(128)
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16, device=DEV)
    qo, ko = pda.rope(e, e, torch.empty(0, dtype=torch.int64, device=DEV), f)
    assert qo.shape == e.shape
    with pytest.raises(pda.PdaError):
        pda.rope(torch.zeros(1, 1, 128, dtype=torch.bfloat16), None, torch.zeros(1, dtype=torch.int64), f)


@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("lengths,first,bs", [([700, 333, 470], 0, 16), ([900], 5, 64), ([611, 600], 40, 48)])
def test_runs_that_start_off_the_slot_grid(lengths, first, bs, shuffled):
    # packed prompts, and a chunk that goes on inside a block: the same bytes as token by token
    H, Hk, T = 8, 8, sum(lengths)
    qkv, pos = inputs(T, H, Hk, seed=T)
    per = [-(-(first + n) // bs) for n in lengths]
    NB = sum(per) + 2
    blocks = torch.randperm(NB, generator=torch.Generator().manual_seed(1))
    slots = torch.cat([blocks[sum(per[:i]):][(first + torch.arange(n)) // bs] * bs + (first + torch.arange(n)) % bs
                       for i, n in enumerate(lengths)])
    f = pda.rope_frequencies(128)[0]
    q, k, v = split(qkv.to(DEV), H, Hk)
    pos, slots = pos.to(DEV), slots.to(DEV)
    shape = (NB, Hk, bs // 16, 128, 16) if shuffled else (NB, Hk, 128, bs)
    caches = [[torch.full(s, 0x55, dtype=torch.uint8, device=DEV) for s in ((NB, Hk, 8, bs, 16), shape)] for _ in range(2)]
    a = pda.rope_and_cache(q, k, v, pos, slots, f, *caches[0], 0.05, 0.03, v_shuffled=shuffled)
    b = torch.cat([pda.rope_and_cache(q[t:t + 1], k[t:t + 1], v[t:t + 1], pos[t:t + 1], slots[t:t + 1], f, *caches[1],
                                      0.05, 0.03, v_shuffled=shuffled) for t in range(T)])
    assert pda.query_device_status() == 0
    assert torch.equal(a, b) and torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])
