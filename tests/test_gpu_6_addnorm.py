"""GPU tests of the residual addition + RMSNorm + 1x128 quantization and of its
backward.  The forward equals the separate addition and the RMSNorm quantizer
(and the CPU oracle) bit for bit; the backward is compared with its formula in
64 bits within first-order rounding bounds, and with differences."""
import pytest
import torch

import oracle
from tests.gpu_util import assert_codes_equal, assert_scales_equal, bits

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def jet(torch_cuda):
    import fp8_block_quantized_gb300 as j
    j.load()
    return j


def stream_pair(M, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    x[:, torch.randperm(K, generator=g)[:max(1, K // 500)]] *= 50.0
    d = torch.randn((M, K), generator=g) * 0.5
    gain = 1 + 0.1 * torch.randn((K,), generator=g)
    return x.to(BF16), d.to(BF16), gain.to(BF16)


SHAPES = [(1, 128), (1, 4096), (2, 256), (7, 384), (16, 5120), (33, 1024), (150, 2048), (153, 8192),
          (305, 4096), (700, 640), (1217, 8320), (3, 14336), (5, 24576), (40, 25600), (2, 65536), (5000, 128)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("eps", [1e-5, 0.0])
def test_equals_the_separate_operators(jet, M, K, eps):
    x, d, g = (t.cuda() for t in stream_pair(M, K, M + K))
    h, q, s, rstd = jet.add_rmsnorm_quant_1x128(x, d, g, eps, with_rstd=True)
    href = (x.float() + d.float()).to(BF16)
    qr, sr = jet.rmsnorm_quant_1x128(href, g, eps)
    torch.cuda.synchronize()
    assert torch.equal(h.view(torch.int16), href.view(torch.int16))
    assert torch.equal(q, qr)
    assert torch.equal(s.view(torch.int32), sr.view(torch.int32))
    ref = 1 / (href.double().square().mean(1) + eps).sqrt()
    # K / 32 additions in a lane, five levels, then four operations, each 2^-24; the root halves the sum's
    assert ((rstd.double() - ref).abs() <= (K / 64 + 8.5) * 2.0 ** -24 * ref).all()


@pytest.mark.parametrize("M,K", [(1, 256), (37, 640), (16, 4096), (310, 1280)])
def test_against_the_oracle(jet, M, K):
    x, d, g = stream_pair(M, K, 5 * M + K)
    h, q, s = jet.add_rmsnorm_quant_1x128(x.cuda(), d.cuda(), g.cuda(), 1e-6)
    torch.cuda.synchronize()
    qo, so = oracle.rmsnorm_quant_1x128(bits((x.float() + d.float()).to(BF16)), bits(g), 1e-6)
    assert_codes_equal(q, qo)
    assert_scales_equal(s, so)


@pytest.mark.parametrize("M", [1, 9, 400])
@pytest.mark.parametrize("into", ["x", "d"])
def test_in_place(jet, M, into):
    K = 1152
    x, d, g = (t.cuda() for t in stream_pair(M, K, M))
    h, q, s = jet.add_rmsnorm_quant_1x128(x, d, g)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    out = x if into == "x" else d
    jet.jet_add_rmsnorm_quant_1x128(x, d, g, 1e-5, out, q2, s2)
    torch.cuda.synchronize()
    assert torch.equal(out, h) and torch.equal(q2, q) and torch.equal(s2, s)


def test_zero_rows_and_cancellation(jet):
    x, d, g = (t.cuda() for t in stream_pair(6, 512, 3))
    d[1], d[4] = -x[1], -x[4]
    h, q, s, rstd = jet.add_rmsnorm_quant_1x128(x, d, g, 0.0, with_rstd=True)
    torch.cuda.synchronize()
    for r in (1, 4):
        assert (h[r] == 0).all() and rstd[r] == 0 and (s[:, r] == 1).all()
        assert ((q[r] & 0x7F) == 0).all()
    assert (rstd[[0, 2, 3, 5]] > 0).all()


def test_empty(jet):
    e = torch.empty((0, 256), dtype=BF16, device="cuda")
    g = torch.ones((256,), dtype=BF16, device="cuda")
    h, q, s = jet.add_rmsnorm_quant_1x128(e, e, g)
    assert h.shape == (0, 256) and s.shape == (2, 0)
    dx, dg = jet.add_rmsnorm_bwd(e, g, torch.empty((0,), device="cuda"), [e])
    torch.cuda.synchronize()
    assert dx.shape == (0, 256) and (dg == 0).all()


# ---------------------------------------------------------------- backward

def bwd_inputs(M, K, n, dres, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda std: (torch.randn((M, K), generator=g) * std).to(BF16).cuda()
    h, gain = r(1.5), (1 + 0.1 * torch.randn((K,), generator=g)).to(BF16).cuda()
    rstd = (1 / (h.double().square().mean(1) + 1e-5).sqrt()).float()
    return h, gain, rstd, [r(1e-2) for _ in range(n)], r(1e-2) if dres else None


def bwd_ref(h, g, rstd, dys, dres):
    """The formula in 64 bits, and the magnitudes its rounding errors scale with."""
    K = h.shape[1]
    r, dy = rstd.double()[:, None], sum(t.double() for t in dys)
    mag_dy = sum(t.double().abs() for t in dys)
    xh, u = h.double() * r, dy * g.double()
    a = (u * xh).sum(1, keepdim=True) / K
    mag_u = mag_dy * g.double().abs()
    mag_a = (mag_u * xh.abs()).sum(1, keepdim=True) / K
    dx, mag = r * (u - xh * a), r * (mag_u + xh.abs() * mag_a)
    if dres is not None:
        dx, mag = dx + dres.double(), mag + dres.double().abs()
    return dx, mag, (dy * xh).sum(0), (mag_dy * xh.abs()).sum(0)


def check_bwd(jet, h, g, rstd, dys, dres, dx, dg):
    M, K = h.shape
    rdx, mag, rdg, mag_dg = bwd_ref(h, g, rstd, dys, dres)
    # binary32 steps: 2 sums of dy, 2 products, at most 32 terms of a thread, 10 levels of shuffles,
    # the division and 3 operations: below 64 in all; one rounding to BF16
    assert ((dx.double() - rdx).abs() <= 2.0 ** -8 * rdx.abs() + 64 * 2.0 ** -24 * mag).all()
    # dy (2), its product with xh (2), rows of one partial, at most 38 partials of a group, 8 groups
    steps = 4 + -(-M // 152) + 38 + 8
    assert ((dg.double() - rdg).abs() <= steps * 2.0 ** -24 * mag_dg).all()


@pytest.mark.parametrize("M,K", [(1, 128), (1, 4096), (3, 384), (16, 5120), (77, 8192), (305, 1024),
                                 (700, 4096), (1537, 640), (5, 8320), (9, 16384), (2, 32768),
                                 (4099, 256)])
@pytest.mark.parametrize("n,dres", [(1, False), (1, True), (2, True), (3, True), (3, False)])
def test_backward(jet, M, K, n, dres):
    h, g, rstd, dys, dr = bwd_inputs(M, K, n, dres, M * 7 + K + n)
    dx, dg = jet.add_rmsnorm_bwd(h, g, rstd, dys, dr)
    torch.cuda.synchronize()
    check_bwd(jet, h, g, rstd, dys, dr, dx, dg)


@pytest.mark.parametrize("M,K", [(400, 8320), (333, 12288), (200, 16384), (170, 16512), (160, 20480), (9, 28672),
                                 (160, 32768)])
@pytest.mark.parametrize("n,dres", [(1, False), (2, True), (3, True)])
def test_backward_of_long_rows(jet, M, K, n, dres):
    """Rows of several chunks a thread, several rows a CTA: two, one or none in
    shared memory; in place of the residual's gradient too."""
    h, g, rstd, dys, dr = bwd_inputs(M, K, n, dres, M + K + n)
    dx, dg = jet.add_rmsnorm_bwd(h, g, rstd, dys, dr)
    torch.cuda.synchronize()
    check_bwd(jet, h, g, rstd, dys, dr, dx, dg)
    if dres:
        dg2 = torch.empty_like(dg)
        jet.jet_add_rmsnorm_bwd(h, g, rstd, dys, dr, dr, dg2)
        torch.cuda.synchronize()
        assert torch.equal(dr, dx) and torch.equal(dg, dg2)


def test_backward_in_place_and_repeatable(jet):
    h, g, rstd, dys, dr = bwd_inputs(1000, 1024, 3, True, 1)
    dx, dg = jet.add_rmsnorm_bwd(h, g, rstd, dys, dr)
    dg2 = torch.empty_like(dg)
    jet.jet_add_rmsnorm_bwd(h, g, rstd, dys, dr, dr, dg2)
    torch.cuda.synchronize()
    assert torch.equal(dr, dx) and torch.equal(dg, dg2)


def test_backward_of_zero_rows(jet):
    h, g, rstd, dys, dr = bwd_inputs(5, 256, 2, True, 2)
    rstd[2] = 0.0                                   # what the forward writes for a zero row at eps 0
    dx, dg = jet.add_rmsnorm_bwd(h, g, rstd, dys, dr)
    torch.cuda.synchronize()
    assert torch.equal(dx[2], dr[2])
    check_bwd(jet, h, g, rstd, dys, dr, dx, dg)


def test_backward_against_differences(jet):
    """Directional derivatives of sum(w y) + sum(v h), y the binary64 norm, by
    central differences: error of the difference ~ step^2, of dx as bounded above."""
    M, K, eps, step = 4, 256, 1e-5, 1e-5
    h, g, _, (w,), v = bwd_inputs(M, K, 1, True, 3)
    rstd = (1 / (h.double().square().mean(1) + eps).sqrt()).float()
    dx, dg = jet.add_rmsnorm_bwd(h, g, rstd, [w], v)
    torch.cuda.synchronize()

    def loss(hh, gg):
        y = hh * gg / (hh.square().mean(1, keepdim=True) + eps).sqrt()
        return (w.double() * y).sum() + (v.double() * hh).sum()
    gen = torch.Generator().manual_seed(4)
    _, mag, _, mag_dg = bwd_ref(h, g, rstd, [w], v)
    for _ in range(8):
        t = torch.randn((M, K), generator=gen, dtype=torch.float64).cuda()
        num = (loss(h.double() + step * t, g.double()) - loss(h.double() - step * t, g.double())) / (2 * step)
        got = (dx.double() * t).sum()
        bound = (t.abs() * (2.0 ** -8 * dx.double().abs() + 64 * 2.0 ** -24 * mag)).sum()
        assert abs(num - got) <= bound + 1e-7
        t = torch.randn((K,), generator=gen, dtype=torch.float64).cuda()
        num = (loss(h.double(), g.double() + step * t) - loss(h.double(), g.double() - step * t)) / (2 * step)
        assert abs(num - (dg.double() * t).sum()) <= (t.abs() * 54 * 2.0 ** -24 * mag_dg).sum() + 1e-7


def test_on_a_side_stream_and_in_a_graph(jet):
    x, d, g = (t.cuda() for t in stream_pair(64, 1024, 9))
    ref = jet.add_rmsnorm_quant_1x128(x, d, g)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = jet.add_rmsnorm_quant_1x128(x, d, g, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    h, q, s = (torch.zeros_like(t) for t in ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jet.jet_add_rmsnorm_quant_1x128(x, d, g, 1e-5, h, q, s)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, (h, q, s)))
