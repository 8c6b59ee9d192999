"""GPU tests of the rotary positions: against the formula in 64 bits, the
backward as its transpose, and the fused KV-cache write against the separate
calls bit for bit."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64


@pytest.fixture(scope="module")
def jet(torch_cuda):
    import fp8_block_quantized_gb300 as j
    j.load()
    return j


def heads(T, H, D, seed, pad=0):
    """[T, H, D] view of rows of H*D + pad elements."""
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn((T, H * D + pad), generator=g).to(BF16).cuda()
    return rows[:, :H * D].unflatten(1, (H, D))


def freqs(R, base=10000.0):
    return (base ** (-torch.arange(0, R, 2, dtype=F64) / max(R, 1))).cuda()


def ref_rope(x, f, pos, layout, mscale, backward):
    """(result, |a| + |b| of each channel's pair) in 64 bits; whole turns are
    taken out with exact integers, so any position is a fair one."""
    R = 2 * f.numel()
    turns = [[math.fmod(int(p) * float(v) / (2 * math.pi), 1.0) for v in f.tolist()] for p in pos.tolist()]
    a = 2 * math.pi * torch.tensor(turns, dtype=F64).reshape(len(turns), R // 2).cuda()[:, None]
    c, s = torch.cos(a) * mscale, torch.sin(a) * mscale * (-1 if backward else 1)
    y, mag = x.double().clone(), torch.zeros(x.shape, dtype=F64, device="cuda")
    i = torch.arange(R // 2, device="cuda")
    ia, ib = (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)
    xa, xb = x.double()[..., ia], x.double()[..., ib]
    y[..., ia], y[..., ib] = xa * c - xb * s, xb * c + xa * s
    mag[..., ia] = mag[..., ib] = (xa.abs() + xb.abs()) * abs(mscale)
    return y, mag


def check(got, x, f, pos, layout, mscale=1.0, backward=False):
    y, mag = ref_rope(x, f, pos, layout, mscale, backward)
    # the reference's angle: pos f (1 + 2^-52); the kernel's: its top 32 bits (2^-31 half turns) and their
    # rounding to binary32 (2^-25 pi radians), sin and cos within 2 ulps, two products and a sum
    angle = pos.double().abs()[:, None, None] * 2.0 ** -50 + 2.0 ** -23
    bound = 2.0 ** -8 * y.abs() + (angle + 6 * 2.0 ** -24) * mag
    err = (got.double() - y).abs()
    assert (err <= bound).all(), (err - bound).max()
    R = 2 * f.numel()
    assert torch.equal(got[..., R:], x[..., R:])           # channels past R are copied


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hk,D,R", [
    (1, 1, 1, 8, 8), (1, 32, 8, 128, 128), (5, 4, 2, 64, 32), (33, 3, 1, 80, 80), (7, 2, 1, 128, 34),
    (3, 5, 5, 96, 2), (129, 8, 2, 256, 128), (4, 2, 2, 48, 0), (2, 1, 1, 1024, 1024), (600, 16, 4, 64, 64),
    (1000, 40, 8, 128, 96), (2, 3, 2, 24, 24), (300, 7, 3, 40, 22)])
def test_forward_and_backward(jet, layout, T, Hq, Hk, D, R):
    q, k = heads(T, Hq, D, T + D), heads(T, Hk, D, T + D + 1, pad=8)
    f = freqs(R)
    g = torch.Generator().manual_seed(R)
    pos = torch.randint(0, 5000, (T,), generator=g).cuda()
    for backward in (False, True):
        qo, ko = jet.rope(q, k, f, pos, layout, 1.0, backward)
        torch.cuda.synchronize()
        check(qo, q, f, pos, layout, 1.0, backward)
        check(ko, k, f, pos, layout, 1.0, backward)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_and_negative_positions(jet, layout):
    pos = torch.tensor([0, 1, -1, 2047, 131071, 1 << 20, (1 << 24) + 1, -(1 << 22), 10 ** 8]).cuda()
    q, f = heads(9, 4, 128, 1), freqs(128, 500000.0)
    qo, _ = jet.rope(q, None, f, pos, layout)
    torch.cuda.synchronize()
    check(qo, q, f, pos, layout)
    assert torch.equal(qo[0], q[0])                         # position 0 is the identity


@pytest.mark.parametrize("layout,R", [("half", 64), ("interleaved", 64), ("half", 36), ("interleaved", 36)])
def test_in_place_strided_and_scaled(jet, layout, R):
    T, Hq, Hk, D = 65, 6, 2, 64
    rows = torch.randn((T, (Hq + Hk) * D + 16), generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    q = rows[:, :Hq * D].unflatten(1, (Hq, D))
    k = rows[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    f, pos = freqs(R), torch.arange(100, 100 + T).cuda()
    qr, kr = jet.rope(q, k, f, pos, layout, 1.25)
    before, tail = rows.clone(), rows[:, (Hq + Hk) * D:].clone()
    jet.jet_rope(q, k, f, pos, q, k, layout, 1.25)
    torch.cuda.synchronize()
    assert torch.equal(q, qr) and torch.equal(k, kr)
    assert torch.equal(rows[:, (Hq + Hk) * D:], tail)       # the row's other elements stay
    check(q, before[:, :Hq * D].unflatten(1, (Hq, D)), f, pos, layout, 1.25)


def test_backward_is_the_transpose(jet):
    """<dy, rope(x)> = <rope_backward(dy), x> up to the two BF16 roundings."""
    T, H, D = 50, 4, 128
    x, dy = heads(T, H, D, 5), heads(T, H, D, 6)
    f, pos = freqs(96), torch.arange(T).cuda() * 37
    y, _ = jet.rope(x, None, f, pos, "half", 1.1)
    dx, _ = jet.rope(dy, None, f, pos, "half", 1.1, backward=True)
    torch.cuda.synchronize()
    a, b = (dy.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    bound = (2.0 ** -8 + 2.0 ** -20) * ((dy.double() * y.double()).abs().sum() + (dx.double() * x.double()).abs().sum())
    assert abs(a - b) <= bound


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hk,D,R", [(1, 32, 8, 128, 128), (64, 8, 8, 64, 64), (37, 4, 1, 80, 22),
                                         (9, 0, 2, 128, 64), (500, 64, 8, 128, 128), (6, 3, 3, 16, 16),
                                         (3, 2, 2, 256, 0), (2000, 4, 4, 96, 96)])
def test_fused_write_equals_the_separate_calls(jet, layout, T, Hq, Hk, D, R):
    S = 2 * T + 3
    q, k, v = heads(T, Hq, D, 1), heads(T, Hk, D, 2, pad=16), heads(T, Hk, D, 3, pad=8)
    g = torch.Generator().manual_seed(T)
    f, pos = freqs(R, 500000.0), torch.randint(0, 100000, (T,), generator=g).cuda()
    slots = torch.randperm(S, generator=g)[:T]
    if T > 5:
        slots[3], slots[5] = -1, S + 7                       # padding and a slot past the cache
    slots = slots.cuda()
    ks = (torch.rand((Hk,), generator=g) * 0.01 + 0.003).cuda()   # some entries saturate
    vs = (torch.rand((Hk,), generator=g) * 0.01 + 0.003).cuda()
    if Hk > 1:
        vs[1] = 2.0 ** -95                                   # the exact slow division
    kc, vc = (torch.full((S, Hk, D), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2))
    kc2, vc2 = kc.clone(), vc.clone()
    qo = torch.empty((T, Hq, D), dtype=BF16, device="cuda")
    jet.jet_rope_kv_cache_write(q, k, v, f, pos, ks, vs, slots, qo, kc, vc, layout, 1.0)
    kr, qr = jet.rope(k, q if Hq else None, f, pos, layout)
    jet.jet_kv_cache_write(kr.contiguous(), ks, slots, kc2)
    jet.jet_kv_cache_write(v.contiguous(), vs, slots, vc2)
    torch.cuda.synchronize()
    if Hq:
        assert torch.equal(qo, qr)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hk,D,R", [(70, 5, 2, 72, 32), (70, 5, 2, 72, 64), (70, 3, 1, 88, 16), (9, 2, 1, 8, 8),
                                         (33, 4, 4, 24, 0), (2500, 9, 3, 128, 64), (2500, 7, 2, 256, 130),
                                         (1300, 32, 8, 128, 128), (40, 3, 2, 1024, 514), (40, 3, 2, 1024, 1022),
                                         (5, 9, 1, 512, 510), (700, 40, 8, 16, 14), (300, 100, 20, 64, 2),
                                         (5000, 17, 3, 128, 34)])
def test_channels_past_the_turned_ones(jet, layout, T, Hq, Hk, D, R):
    """Odd numbers of chunks past R, heads that no thread's batch divides, in
    numbers that take several rounds of the grid."""
    q, k = heads(T, Hq, D, T + D), heads(T, Hk, D, T + D + 1, pad=8)
    f, pos = freqs(max(R, 2))[:R // 2], torch.arange(T).cuda() * 3
    for backward in (False, True):
        qo, ko = jet.rope(q, k, f, pos, layout, 1.0, backward)
        torch.cuda.synchronize()
        check(qo, q, f, pos, layout, 1.0, backward)
        check(ko, k, f, pos, layout, 1.0, backward)
        assert torch.equal(qo[:, :, R:], q[:, :, R:]) and torch.equal(ko[:, :, R:], k[:, :, R:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hk,D,R", [(1700, 32, 8, 128, 128), (1700, 32, 8, 128, 64), (3000, 9, 3, 80, 48),
                                         (2600, 13, 1, 256, 128), (6000, 7, 1, 96, 26), (20000, 2, 1, 64, 64), (5000, 17, 3, 128, 34),
                                         (50, 3, 2, 1024, 514), (900, 40, 24, 16, 14)])
def test_fused_write_of_many_tokens(jet, layout, T, Hq, Hk, D, R):
    """Equal to the two separate calls where a thread takes its heads in twos."""
    S = T + 7
    q, k, v = heads(T, Hq, D, 1), heads(T, Hk, D, 2, pad=16), heads(T, Hk, D, 3, pad=8)
    g = torch.Generator().manual_seed(T)
    f, pos = freqs(R, 500000.0), torch.randint(0, 100000, (T,), generator=g).cuda()
    slots = torch.randperm(S, generator=g)[:T].cuda()
    slots[11] = -1
    ks, vs = ((torch.rand((Hk,), generator=g) * 0.01 + 0.003).cuda() for _ in range(2))
    kc, vc = (torch.full((S, Hk, D), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2))
    kc2, vc2 = kc.clone(), vc.clone()
    qo, ko = jet.rope(q, k, f, pos, layout, 1.1)
    jet.jet_kv_cache_write(ko, ks, slots, kc2)
    jet.jet_kv_cache_write(v.contiguous(), vs, slots, vc2)
    qf = torch.empty((T, Hq, D), dtype=BF16, device="cuda")
    jet.jet_rope_kv_cache_write(q, k, v, f, pos, ks, vs, slots, qf, kc, vc, layout, 1.1)
    torch.cuda.synchronize()
    assert torch.equal(qf, qo) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


@pytest.mark.parametrize("R", [64, 36])
def test_no_heads_to_cache(jet, R):
    """With Hk = 0 nothing of the cache's is read: its pointers and the slots may be null."""
    T, H, D = 33, 4, 64
    q, f, pos = heads(T, H, D, 3), freqs(R), torch.arange(T).cuda()
    want, _ = jet.rope(q, None, f, pos, "half", 1.2)
    out = torch.empty((T, H, D), dtype=BF16, device="cuda")
    st = jet.load().jet_rope_kv_cache_write(
        q.data_ptr(), q.stride(0), H, None, 0, None, 0, 0, T, D, R, f.data_ptr(), pos.data_ptr(), 0, 1.2,
        None, None, None, out.data_ptr(), H * D, None, None, 0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(out, want)


def test_cache_past_32_bits(jet):
    """Slots whose byte offsets pass 2^32 land where they belong."""
    T, H, D = 3, 8, 128
    S = (1 << 32) // (H * D) + 5
    kc = torch.zeros((S, H, D), dtype=torch.uint8, device="cuda")
    vc = torch.zeros((S, H, D), dtype=torch.uint8, device="cuda")
    q, k, v = (heads(T, H, D, i) for i in range(3))
    slots = torch.tensor([S - 1, 0, S - 4]).cuda()
    ones = torch.full((H,), 0.02, device="cuda")
    f, pos = freqs(D), torch.arange(T).cuda()
    jet.jet_rope_kv_cache_write(q, k, v, f, pos, ones, ones, slots, torch.empty_like(q), kc, vc)
    small = torch.zeros((T, H, D), dtype=torch.uint8, device="cuda")
    small_v = torch.zeros_like(small)
    jet.jet_rope_kv_cache_write(q, k, v, f, pos, ones, ones, torch.arange(T).cuda(), torch.empty_like(q),
                                small, small_v)
    torch.cuda.synchronize()
    assert torch.equal(kc[slots], small) and torch.equal(vc[slots], small_v)
    assert int(kc[S - 2].sum()) == 0 and int(kc[1].sum()) == 0


def test_empty(jet):
    e = torch.empty((0, 4, 64), dtype=BF16, device="cuda")
    q, k = jet.rope(e, e, freqs(64), torch.empty((0,), dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    assert q.shape == (0, 4, 64)


def test_more_tokens_than_one_launch_counts(jet):
    """2^30 tokens of one small head (items past 32 bits, offsets past 2^33 bytes):
    the last tokens are turned as in a small call, the others keep their zeros."""
    T, D, at = (1 << 30) + 5, 8, [0, 3, (1 << 30) - 1, 1 << 30, (1 << 30) + 4]
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 40 GB")
    f = freqs(D)
    q = torch.zeros((T, 1, D), dtype=BF16, device="cuda")
    pos = torch.arange(T, device="cuda")
    rows = heads(len(at), 1, D, 3)
    at = torch.tensor(at, device="cuda")
    q[at] = rows
    jet.jet_rope(q, None, f, pos, q, None)
    small, _ = jet.rope(rows, None, f, pos[at])
    torch.cuda.synchronize()
    assert torch.equal(q[at], small)
    q[at] = 0
    assert not q.any()
