"""GPU tests of the attention over the paged cache where single values decide:
NaN codes and scales, weights far below a row's largest, indexes past 32 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F8, F32, F64, I32, I64, U8 = (torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.float64,
                                    torch.int32, torch.int64, torch.uint8)
INF = float("inf")


@pytest.fixture(scope="module")
def jet(torch_cuda):
    import fp8_block_quantized_gb300 as j
    j.load()
    return j


def codes(x):
    return x.clamp(-448, 448).to(F8).view(U8).cuda()


def call(jet, q, k, v, table, bs, new, lengths, ks=None, vs=None, groups=None, scale=1.0):
    """(out, lse) of requests with new[b] tokens each; groups: (offsets, lengths)."""
    T, Hq, D = q.shape
    Hk = k.shape[1]
    one = torch.ones((Hk,), device="cuda")
    out = torch.full((T, Hq, D), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    po, pl = (None, None) if groups is None else (torch.tensor(groups[0]).cuda(),
                                                  torch.tensor(groups[1], dtype=I32).cuda())
    jet.jet_kv_attention(q, k, v, one if ks is None else ks, one if vs is None else vs, table, bs,
                         torch.tensor([0] + new).cumsum(0).cuda(), torch.tensor(lengths, dtype=I32).cuda(),
                         out, lse, po, pl, scale=scale)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("D", [64, 128])
def test_nan_value_in_units_one_behind_another(jet, D):
    """Units of one pair of tiles, some ten for each CTA; the NaN lies in the second tile, which
    all requests share and L2 holds.  The first tiles come from memory and their maxima grow, so
    that their half ends later."""
    Hq, Hk, bs, n, B = 4, 1, 128, 16, 1600
    g = torch.Generator(device="cuda").manual_seed(D)
    k = torch.randn(((B + 1) * bs, Hk, D), generator=g, device="cuda")
    at = torch.arange(bs, device="cuda")
    # 64 keys at a time, the later ones of a tile are weighed first
    k.view(B + 1, bs, D)[:B, :, 0] = torch.where(at < 64, 200.0, -200.0)
    k.view(B + 1, bs, D)[B, :, 0] = -200.0
    v = torch.randn(((B + 1) * bs, Hk, D), generator=g, device="cuda") * 90
    q = torch.randn((B * n, Hq, D), generator=g, device="cuda").to(BF16)
    q[:, :, 0] = 0.25
    table = torch.stack([torch.randperm(B, generator=g, device="cuda"), torch.full((B,), B, device="cuda")], 1)
    args = dict(table=table.to(I32), bs=bs, new=[n] * B, lengths=[2 * bs] * B)
    kc, vc = codes(k), codes(v)
    want, lse = call(jet, q, kc, vc, **args)
    assert torch.isfinite(want.float()).all()
    vc[B * bs + 50, 0, 17] = 0x7F      # every query sees it
    flush = torch.empty((1 << 28,), device="cuda")
    for _ in range(10):
        flush.zero_()
        q.amax(), kc[B * bs:].amax(), vc[B * bs:].amax()
        got, l2 = call(jet, q, kc, vc, **args)
        assert got[:, :, 17].isnan().all(), int((~got[:, :, 17].isnan()).sum())
        assert torch.equal(l2, lse)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 40, 300])       # tokens of a request: few rows a unit, and many
@pytest.mark.parametrize("groups", [None, ([0, 3], [50])])
def test_scales_of_the_keys(jet, D, n, groups):
    """NaN: all queries of the head that see a key, none of another's; zero: the values' mean."""
    Hq, Hk, bs, L = 8, 2, 16, 333
    g = torch.Generator().manual_seed(n)
    S = (L + bs) // bs * bs
    kc, vc = (codes(torch.randn((S, Hk, D), generator=g) * 90) for _ in range(2))
    q = torch.randn((3 * n, Hq, D), generator=g).to(BF16).cuda()
    table = torch.arange(S // bs, dtype=I32).repeat(3, 1).cuda()
    args = dict(table=table, bs=bs, new=[n] * 3, lengths=[L, 0, L], groups=groups, scale=D ** -0.5)
    ks = torch.tensor([0.01, 0.01], device="cuda")
    want, lse = call(jet, q, kc, vc, ks=ks, **args)
    ks[1] = float("nan")
    got, l2 = call(jet, q, kc, vc, ks=ks, **args)
    assert torch.equal(got[:, :4], want[:, :4]) and torch.equal(l2[:, :4], lse[:, :4])
    sees = torch.ones((3 * n,), dtype=torch.bool)
    sees[n:2 * n] = False
    assert got[sees, 4:].isnan().all() and l2[sees, 4:].isnan().all()
    assert not got[~sees].any() and (l2[~sees] == -INF).all()
    ks[1] = 0.0
    got, l2 = call(jet, q, kc, vc, ks=ks, **args)
    v = vc.view(F8).double()[:, 1]
    mean = v.cumsum(0) / torch.arange(1, S + 1, device="cuda")[:, None]
    size = v.abs().cumsum(0) / torch.arange(1, S + 1, device="cuda")[:, None]
    for t in list(range(n)) + list(range(2 * n, 3 * n)):
        seen = L - n + t % n + 1
        # weights of 1 up to the factor's floor (2^-126 of a raw score: nothing); sums of `seen` terms in
        # binary32, and the output's rounding
        bound = 2.0 ** -8 * mean[seen - 1].abs() + 2 * (seen + 8) * 2.0 ** -24 * size[seen - 1]
        assert ((got[t, 4:].double() - mean[seen - 1]).abs() <= bound).all()
        assert ((l2[t, 4:].double() - math.log(seen)).abs() <= (seen + 16) * 2.0 ** -24).all()


def test_more_tiles_than_32_bits_count(jet):
    """A group of more than 2^32 tiles of 8 rows and 32 keys, of which all but the first few have
    no slot."""
    Hq, Hk, D, bs, T, width = 256, 1, 64, 1 << 16, 1040, 64
    assert T * Hq // 8 * (width * bs // 32) > 2 ** 32
    g = torch.Generator().manual_seed(5)
    kc, vc = (codes(torch.randn((100, Hk, D), generator=g) * 90) for _ in range(2))
    q = torch.randn((T, Hq, D), generator=g).to(BF16).cuda()
    table = torch.full((1, width), -1, dtype=I32, device="cuda")
    table[0, 0] = 0                                # keys 0 .. 99; slots behind them are not there
    ks = torch.full((Hk,), 0.01, device="cuda")
    args = dict(table=table, bs=bs, new=[T], ks=ks, scale=D ** -0.5)
    out, lse = call(jet, q, kc, vc, lengths=[width * bs], groups=([0, 1], [width * bs - T]), **args)
    k, v = kc.view(F8).double()[:, 0] * ks.double(), vc.view(F8).double()[:, 0]
    x = q.double() @ k.t() * D ** -0.5                                       # [T, Hq, 100]
    w = torch.softmax(x, 2)
    ref = w @ v
    # a score: D products summed in binary32 and the factor's roundings, e^x to 2^-22; a weight: that twice
    # and FP16's 2^-11 (or 2^-25 of the largest); sums of 100 terms and the joins' in binary32; BF16's 2^-8.
    # (Another split of the keys among workers gives other roundings: no call is bit for bit another's.)
    dx = (D + 8) * 2.0 ** -24 * (q.double().abs() @ k.abs().t()).amax(2) * D ** -0.5 + 2.0 ** -22 * x.abs().amax(2)
    rel = 2.0 ** -11 + 2 * dx + 2.0 ** -21 + 300 * 2.0 ** -24
    bound = 2.0 ** -8 * ref.abs() + rel[..., None] * (w @ v.abs()) + 2.0 ** -25 * v.abs().sum(0) * w.amax(2)[..., None]
    assert ((out.double() - ref).abs() <= bound).all()
    rl = torch.logsumexp(x, 2)
    assert ((lse.double() - rl).abs() <= dx + 2.0 ** -21 + 300 * 2.0 ** -24 + 2.0 ** -22 * rl.abs()).all()
