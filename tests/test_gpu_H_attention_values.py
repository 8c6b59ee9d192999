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


def sink(n, G, D, gap, L, seed):
    """(q, k, v, k_scale): L keys of score 0, and key 100 of score `gap`, whose values are zero."""
    g = torch.Generator().manual_seed(seed)
    k = torch.zeros((L, 1, D))
    k[100, 0, 0] = 448
    kc = codes(k)
    v = torch.rand((L, 1, D), generator=g) * 400 + 40
    v[100] = 0
    vc = codes(v)
    q = torch.randn((n, G, D), generator=g).to(BF16).cuda()
    q[:, :, 0] = 1.0
    return q, kc, vc, torch.tensor([gap / 448], device="cuda")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,n,B", [(4, 1, 2048), (8, 16, 304), (4, 64, 304)])   # rows of a unit: 4, 128, 256
@pytest.mark.parametrize("gap", [15.0, 17.0, 18.0, 20.0])
def test_keys_far_below_the_largest(jet, D, G, n, B, gap):
    """One key without values far above 8191 others, all in one piece: they are the output."""
    L = 8192
    q, kc, vc, ks = sink(n, G, D, gap, L, int(gap) + n)
    table = torch.arange(L // 64, dtype=I32).repeat(B, 1).cuda()
    out, lse = call(jet, q.repeat(B, 1, 1), kc, vc, table, 64, [n] * B, [L] * B, ks=ks)
    x = float(ks) * 448
    v = vc.view(F8).double()[:, 0]
    seen = torch.arange(L - n, L, device="cuda") + 1
    total = v.cumsum(0)[seen - 1]                                             # [n, D]
    e = math.exp(-x)
    z = 1 + (seen - 1) * e
    ref = (e * total / z[:, None])[:, None]                                   # [n, 1, D]
    # scores are exact but for the factor's roundings and the argument's (2^-22 x in all); a weight: that,
    # e^x to 2^-22, FP16's 2^-11, and 2^-32 of the largest near its smallest; sums of L terms, cut off or
    # rounded 16 at a time; BF16's 2^-8
    rel = 2.0 ** -8 + 2.0 ** -11 + 2 * (2.0 ** -22 * x + 2.0 ** -22) + 2 * L * 2.0 ** -24
    bound = rel * ref + 2.0 ** -32 * total[:, None] / z[:, None, None]
    got = out.view(B, n, G, D).double()
    assert ((got - ref).abs() <= bound).all(), ((got - ref).abs() / ref).max()
    rl = x + torch.log(z)
    assert ((lse.view(B, n, G).double() - rl[:, None]).abs() <= 2.0 ** -20 + 2.0 ** -22 * x + L * 2.0 ** -24).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,n", [(4, 1), (8, 16), (4, 64)])
@pytest.mark.parametrize("power", [10, 17, 19, 20, 21, 24, 26])
def test_large_scores(jet, D, G, n, power):
    """Scores whose own rounding is up to four powers of two: the largest one's value alone."""
    B, L = 3, 1500
    for gap in (1.1 * 2 ** power, 1.37 * 2 ** power, -1.77 * 2 ** power):
        q, kc, vc, ks = sink(n, G, D, abs(gap), L, power)
        if gap < 0:                          # all others share the largest score, 0
            kc[100, 0, 0] |= 0x80
        else:
            vc[100] = vc[99]
        table = torch.arange((L + 63) // 64, dtype=I32).repeat(B, 1).cuda()
        pad = 64 * table.shape[1] - L
        kc, vc = (torch.cat([c, c[:pad]]) for c in (kc, vc))
        out, lse = call(jet, q.repeat(B, 1, 1), kc, vc, table, 64, [n] * B, [L] * B, ks=ks)
        v = vc.view(F8).double()[:, 0]
        seen = torch.arange(L - n, L, device="cuda") + 1
        x = float(ks) * 448
        if gap > 0:
            ref, rl = v[100].expand(n, D), torch.full((n,), x, dtype=F64, device="cuda")
        else:
            ref, rl = v.cumsum(0)[seen - 1] / (seen - 1)[:, None], torch.log((seen - 1).double())
        # weights that are equal are rounded alike (2^-11), sums of L terms, BF16
        got = out.view(B, n, G, D).double()
        assert ((got - ref[:, None]).abs() <= (2.0 ** -8 + 2.0 ** -11 + 2 * L * 2.0 ** -24) * ref[:, None]).all()
        assert ((lse.view(B, n, G).double() - rl[:, None]).abs() <= 2.0 ** -22 * rl[:, None] + 2.0 ** -20 + L * 2.0 ** -24).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,n,B", [(4, 1, 2048), (8, 16, 304), (4, 64, 304)])   # a unit in one piece
@pytest.mark.parametrize("power", [20, 25, 26])
def test_large_scores_beside_each_other(jet, D, G, n, B, power):
    """Two keys whose scores are the same value or neighbouring ones, in one tile and the next, and
    whose values are the same: their order and distance do not show."""
    L = 900
    for step, gap in [(s, 1.37 + j / 64) for s in (0, 2, 4) for j in range(12)]:
        q, kc, vc, ks = sink(n, G, D, gap * 2 ** power, L, step)
        q[:, :, 1] = 2.0 ** -22                     # a unit of key 500's second channel: 2^-22 of the first's
        kc[500] = kc[100]
        kc[500, 0, 1] = codes(torch.tensor([64.0 * step]))[0]
        vc[100] = vc[99]
        vc[500] = vc[99]
        table = torch.arange((L + 63) // 64, dtype=I32).repeat(B, 1).cuda()
        pad = 64 * table.shape[1] - L
        kc, vc = (torch.cat([c, c[:pad]]) for c in (kc, vc))
        for swap in (False, True):
            if swap:
                kc[[100, 500]] = kc[[500, 100]]
            out, _ = call(jet, q.repeat(B, 1, 1), kc, vc, table, 64, [n] * B, [L] * B, ks=ks)
            v = vc.view(F8).double()[99, 0]
            # the others' weights are zero; two weights of any sizes, each rounded to 2^-11, BF16
            assert ((out.double() - v).abs() <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -21) * v).all()
