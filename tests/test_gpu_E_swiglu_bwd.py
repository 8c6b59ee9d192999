"""GPU tests of the gated activation's backward with its quantization: against
the formula in 64 bits, and against differences."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def jet(torch_cuda):
    import fp8_block_quantized_gb300 as j
    j.load()
    return j


def gradients(gate, up, dh):
    g, u, d = (t.double() for t in (gate, up, dh))
    s, c = torch.sigmoid(g), torch.sigmoid(-g)
    # the relative error of each factor: e^-|g| 2^-22 + |g| 2^-24 (its argument's rounding), the
    # reciprocal 2^-23, three products 2^-24 each; 1 + g (1 - s) can cancel, its error is of |g (1 - s)|
    rel = 2.0 ** -20 + g.abs() * 2.0 ** -23
    dup, base = d * g * s, d * u * s
    return (base * (1 + g * c), base.abs() * (1 + (g * c).abs()) * rel), (dup, dup.abs() * rel)


def check_form(q, s, value, err):
    M, F = value.shape
    y, e = value.view(M, F // 128, 128), err.view(M, F // 128, 128)
    amax, scale = y.abs().amax(2), s.t().double()
    top = torch.where(amax == 0, 1.0, amax / 448)
    assert ((scale - top).abs() <= e.amax(2) / 448 + 2.0 ** -24 * top + 2.0 ** -149).all()
    got = q.view(F8).double().view(M, F // 128, 128)
    # a code is off by half a step of its own size (2^-4), or of the smallest normal (2^-10)
    x = y / scale[:, :, None]
    bound = 2.0 ** -4 * x.abs().clamp(min=2.0 ** -6) + (e / scale[:, :, None]) * 1.1 + 2.0 ** -20 * x.abs()
    assert ((got - x).abs() <= bound).all(), ((got - x).abs() - bound).max()
    clean = ((x.to(torch.float32).to(F8).double() != got) & (amax > 0)[:, :, None]).double().mean()
    assert clean <= 1e-3                       # and differs from the nearest only beside a border


def check(jet, gate, up, dh):
    qg, sg, qu, su = jet.swiglu_bwd_quant_1x128(gate, up, dh)
    torch.cuda.synchronize()
    a, b = gradients(gate, up, dh)
    check_form(qg, sg, *a)
    check_form(qu, su, *b)
    return qg, sg, qu, su


def rand(M, F, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((M, F), generator=g) * std).to(BF16).cuda()


@pytest.mark.parametrize("M,F", [(1, 128), (3, 384), (128, 256), (129, 1024), (7, 14336), (2000, 640), (4097, 128)])
def test_against_the_formula(jet, M, F):
    check(jet, rand(M, F, 1), rand(M, F, 2), rand(M, F, 3, 1e-3))


def test_views_of_one_product(jet):
    rows = rand(200, 512, 4)
    dh = rand(200, 256, 5)
    got = check(jet, rows[:, :256], rows[:, 256:], dh)
    want = jet.swiglu_bwd_quant_1x128(rows[:, :256].contiguous(), rows[:, 256:].contiguous(), dh)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_range_of_the_gate(jet):
    """Every BF16 gate from -80 to 80 with gradients of several sizes; beyond, where
    e^-|gate| leaves binary32's normal range, only near zero."""
    bits = torch.arange(0, 0x42A1, dtype=torch.int32)          # 0 .. 80
    g = torch.cat([bits, bits + 0x8000]).to(torch.int16).view(BF16)
    F = 128
    g = torch.cat([g, g[:(-g.numel()) % F]]).view(-1, F).cuda()
    for dv in (1.0, 1e-3, 3e8):
        check(jet, g, torch.full_like(g, -1.25), torch.full_like(g, dv))
    far = torch.linspace(-300, 300, 4 * F).to(BF16).view(4, F).cuda()
    one = torch.ones_like(far)
    qg, sg, qu, su = jet.swiglu_bwd_quant_1x128(far, one, one)
    for q, s, (y, _) in zip((qg, qu), (sg, su), gradients(far, one, one)):
        got = q.view(F8).double() * s.t().double().repeat_interleave(128, 1)
        step = 2.0 ** -10 * s.t().double().repeat_interleave(128, 1)
        assert ((got - y).abs() <= 2.0 ** -4 * 1.001 * y.abs() + step + 1e-35).all()


def test_zeros(jet):
    z = torch.zeros((4, 256), dtype=BF16, device="cuda")
    one = torch.ones_like(z)
    for gate, up, dh in ((one, one, z), (z, one, one), (one, z, one)):
        check(jet, gate, up, dh)
    qg, sg, qu, su = jet.swiglu_bwd_quant_1x128(one, one, z)
    assert (sg == 1).all() and (su == 1).all() and not (qg & 0x7F).any() and not (qu & 0x7F).any()


def test_against_differences(jet):
    """The gradients of sum(dh silu(gate) up) by central differences in 64 bits."""
    gate, up, dh = rand(8, 128, 6), rand(8, 128, 7), rand(8, 128, 8)
    f = lambda g, u: dh.double() * g * torch.sigmoid(g) * u
    g, u, h = gate.double(), up.double(), 1e-5
    dg = (f(g + h, u) - f(g - h, u)) / (2 * h)
    du = (f(g, u + h) - f(g, u - h)) / (2 * h)
    qg, sg, qu, su = jet.swiglu_bwd_quant_1x128(gate, up, dh)
    for q, s, d in ((qg, sg, dg), (qu, su, du)):
        got = q.view(F8).double() * s.t().double()
        # half an E4M3 step, of the value or of the smallest normal; differences to 1e-8
        assert ((got - d).abs() <= 2.0 ** -4 * d.abs() * 1.001 + 2.0 ** -10 * s.t().double() + 1e-8).all()


def test_no_rows(jet):
    e = torch.empty((0, 256), dtype=BF16, device="cuda")
    assert jet.swiglu_bwd_quant_1x128(e, e, e)[0].shape == (0, 256)
