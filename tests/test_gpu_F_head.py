"""GPU tests of the head's log-probabilities and their gradient: against the
formulas in 64 bits, and against differences."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def jet(torch_cuda):
    import fp8_block_quantized_gb300 as j
    j.load()
    return j


def make(T, K, V, seed=0, ignored=0.0, std=2.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, K), generator=g).to(BF16).cuda()
    w = (torch.randn((V, K), generator=g) * std * K ** -0.5).to(BF16).cuda()
    target = torch.randint(0, V, (T,), generator=g)
    if ignored:
        gone = torch.rand((T,), generator=g) < ignored
        target[gone] = torch.tensor([-100, -1, V, 2 ** 40])[torch.arange(T) % 4][gone]
    dlogp = torch.randn((T,), generator=g).cuda()
    return x, w, target.cuda(), dlogp


def forward(x, w, target, scale):
    """(z, lse, logp, real, bound of a logit, bound of lse) in 64 bits."""
    T, K = x.shape
    V = w.shape[0]
    z = x.double() @ w.double().t() * scale
    # sums of 16 products at a time into binary32, each step off by a unit of 2^-22 of what was added up
    dz = (x.double().abs() @ w.double().abs().t()).amax(1) * scale * (K / 16 + 2) * 2.0 ** -22
    lse = torch.logsumexp(z, 1)
    real = (target >= 0) & (target < V)
    at = z[torch.arange(T, device="cuda"), torch.where(real, target, 0)]
    # e^x: 2^-22 and its argument's rounding; chains of at most 256 + V / 8192 + 64 sums
    dl = dz + 2.0 ** -22 + z.abs().amax(1) * 2.0 ** -22 + (320 + V / 8192) * 2.0 ** -24
    return z, lse, torch.where(real, at - lse, 0.0), real, dz, dl


SHAPES = [(1, 8, 1), (1, 64, 2), (5, 72, 100), (48, 512, 2048), (127, 128, 127), (128, 520, 128),
          (129, 64, 129), (256, 256, 257), (257, 1024, 1000), (600, 192, 5003), (1, 4096, 20011),
          (130, 2048, 512), (300, 8, 40000)]


@pytest.mark.parametrize("T,K,V", SHAPES)
@pytest.mark.parametrize("scale", [1.0, 1 / 0.7])
def test_logp(jet, T, K, V, scale):
    x, w, target, _ = make(T, K, V, T + K + V, ignored=0.2)
    logp, lse = jet.head_logp(x, w, target, scale)
    torch.cuda.synchronize()
    z, rl, rp, real, dz, dl = forward(x, w, target, scale)
    assert ((lse.double() - rl).abs() <= dl).all(), ((lse.double() - rl).abs() - dl).max()
    assert ((logp.double() - rp).abs() <= dl + dz)[real].all()
    assert (logp[~real] == 0).all()


def check_bwd(x, w, target, dlogp, scale, lse, dx, dw):
    z, _, _, real, dz, _ = forward(x, w, target, scale)
    V = w.shape[0]
    p = torch.exp(z - lse.double()[:, None])
    up = torch.where(real, dlogp.double() * scale, 0.0)
    hot = torch.zeros_like(p)
    rows = torch.nonzero(real)[:, 0]
    hot[rows, target[rows]] = 1.0
    d = torch.where(real[:, None], up[:, None] * (hot - p), 0.0)
    # e^(z - lse): the logit's error, lse's and the argument's roundings; d once more to BF16 (2^-8)
    off = up.abs()[:, None] * p * (2 * dz[:, None] + (z.abs() + lse.double().abs()[:, None] + 8) * 2.0 ** -22)
    off = torch.where(real[:, None], off, 0.0) + 2.0 ** (-16 if len(x) <= 128 else -8) * d.abs()
    for got, ref, bound, n in ((dx, d @ w.double(), off @ w.double().abs(), V),
                               (dw, d.t() @ x.double(), off.t() @ x.double().abs(), x.shape[0])):
        if got is None:
            continue
        mag = (d.abs() @ w.double().abs()) if got is dx else (d.abs().t() @ x.double().abs())
        bound = bound + 2.0 ** -8 * ref.abs() + mag * (n / 16 + 20) * 2.0 ** -22 + 1e-38
        assert ((got.double() - ref).abs() <= bound).all(), ((got.double() - ref).abs() - bound).max()


@pytest.mark.parametrize("T,K,V", SHAPES)
@pytest.mark.parametrize("scale,ignored", [(1.0, 0.0), (1 / 0.7, 0.4)])
def test_gradients(jet, T, K, V, scale, ignored):
    x, w, target, dlogp = make(T, K, V, T + K + V + 1, ignored)
    _, lse = jet.head_logp(x, w, target, scale)
    dx, dw = jet.head_logp_bwd(x, w, target, lse, dlogp, scale)
    torch.cuda.synchronize()
    check_bwd(x, w, target, dlogp, scale, lse, dx, dw)


def test_several_pieces(jet):
    """More tokens than half a gigabyte of d holds a vocabulary for."""
    T, K, V = 66001, 64, 9001
    assert T * V * 2 > (512 << 20)
    x, w, target, dlogp = make(T, K, V, 3, 0.1)
    dlogp /= T
    logp, lse = jet.head_logp(x, w, target)
    _, rl, rp, real, dz, dl = forward(x, w, target, 1.0)
    assert ((lse.double() - rl).abs() <= dl).all() and ((logp.double() - rp).abs() <= dl + dz)[real].all()
    del rl, rp, dl
    dx, dw = jet.head_logp_bwd(x, w, target, lse, dlogp)
    check_bwd(x, w, target, dlogp, 1.0, lse, dx, dw)


def test_one_gradient_alone(jet):
    x, w, target, dlogp = make(70, 128, 999, 4)
    _, lse = jet.head_logp(x, w, target)
    dx, dw = jet.head_logp_bwd(x, w, target, lse, dlogp)
    only = torch.empty_like(dx), torch.empty_like(dw)
    jet.jet_head_logp_bwd(x, w, target, lse, dlogp, 1.0, only[0], None)
    jet.jet_head_logp_bwd(x, w, target, lse, dlogp, 1.0, None, only[1])
    assert torch.equal(only[0], dx) and torch.equal(only[1], dw)


def test_ignored_rows_are_exactly_zero(jet):
    """Whatever their lse and dlogp hold."""
    x, w, target, dlogp = make(40, 64, 300, 5)
    _, lse = jet.head_logp(x, w, target)
    target[::3] = -100
    lse[::3], dlogp[::3] = float("nan"), float("inf")
    dx, dw = jet.head_logp_bwd(x, w, target, lse, dlogp)
    assert not dx[::3].any() and torch.isfinite(dw.float()).all() and dx[1].any()
    target[:] = 300
    dx, dw = jet.head_logp_bwd(x, w, target, lse, dlogp)
    assert not dx.any() and not dw.any()


def test_few_rows_with_a_gradient(jet):
    """The rows without one get exact zeros and add nothing: first, last, single and no rows with one."""
    x, w, target, dlogp = make(700, 128, 1000, 12)
    _, lse = jet.head_logp(x, w, target)
    for keep in ([0], [699], [5, 63, 64, 65, 300], list(range(64)), list(range(100, 229)), []):
        some = torch.zeros((700,), dtype=torch.bool, device="cuda")
        some[keep] = True
        for how in ("target", "dlogp"):
            t2, d2 = target.clone(), dlogp.clone()
            if how == "target":
                t2[~some] = -100
            else:
                d2[~some] = 0.0
            dx, dw = jet.head_logp_bwd(x, w, t2, lse, d2)
            assert not dx[~some].any()
            check_bwd(x, w, t2, d2, 1.0, lse, dx, dw)


def test_one_row_with_a_gradient_many_calls(jet):
    """Few rows of a long contraction and a large vocabulary, calls one behind another."""
    x, w, target, dlogp = make(129, 4096, 32000, 13)
    _, lse = jet.head_logp(x, w, target)
    for keep in (0, 1, 16, 100, 128, 129):
        t2 = target.clone()
        t2[keep:] = -1
        first = jet.head_logp_bwd(x, w, t2, lse, dlogp)
        for _ in range(10):
            dx, dw = jet.head_logp_bwd(x, w, t2, lse, dlogp)
        torch.cuda.synchronize()
        assert jet.device_status()[0] == 0
        assert torch.equal(dx, first[0]) and torch.equal(dw, first[1]) and not dx[keep:].any()
    check_bwd(x, w, target, dlogp, 1.0, lse, dx, dw)


def test_no_tokens(jet):
    x, w, target, dlogp = make(1, 64, 50, 6)
    e = torch.empty((0,), device="cuda")
    assert jet.head_logp(x[:0], w, target[:0])[0].numel() == 0
    dx, dw = jet.head_logp_bwd(x[:0], w, target[:0], e, e)
    assert dx.shape == (0, 64) and not dw.any()


def test_confident_tokens(jet):
    """Targets far above and far below the rest: logp near 0, and very negative."""
    x, w, target, dlogp = make(64, 256, 1000, 7, std=0.5)
    w[target] = 0
    w[target[0]] = (x[0].float() * 0.4).to(BF16)       # one row's target at z of about 100
    w[target[1]] = (x[1].float() * -0.4).to(BF16)
    logp, lse = jet.head_logp(x, w, target)
    _, rl, rp, real, dz, dl = forward(x, w, target, 1.0)
    assert rp[0] > -1e-6 and rp[1] < -50
    assert ((logp.double() - rp).abs() <= dl + dz).all() and (logp <= 0).all()
    dx, dw = jet.head_logp_bwd(x, w, target, lse, dlogp)
    check_bwd(x, w, target, dlogp, 1.0, lse, dx, dw)


def test_against_differences(jet):
    """Directional derivatives of sum(dlogp logp), central differences in 64 bits."""
    x, w, target, dlogp = make(33, 64, 200, 8)
    _, lse = jet.head_logp(x, w, target)
    dx, dw = jet.head_logp_bwd(x, w, target, lse, dlogp)

    def f(a, b):
        z = a @ b.t()
        return (dlogp.double() * (z.gather(1, target[:, None])[:, 0] - torch.logsumexp(z, 1))).sum()
    g = torch.Generator().manual_seed(9)
    xd, wd, h = x.double(), w.double(), 1e-6
    for i in range(4):
        u = torch.randn(x.shape, generator=g, dtype=F64).cuda()
        v = torch.randn(w.shape, generator=g, dtype=F64).cuda()
        # outputs are off by 2^-8 of themselves and d's rounding in them; random directions add up as norms
        for num, grad, way in (((f(xd + h * u, wd) - f(xd - h * u, wd)) / (2 * h), dx, u),
                               ((f(xd, wd + h * v) - f(xd, wd - h * v)) / (2 * h), dw, v)):
            assert abs(num - (grad.double() * way).sum()) <= 2.0 ** -6 * float((grad.double().abs() * way.abs()).sum())


def test_the_same_bits_again_on_another_stream_and_in_a_graph(jet):
    x, w, target, dlogp = make(300, 256, 3001, 10, 0.2)
    logp, lse = jet.head_logp(x, w, target)
    dx, dw = jet.head_logp_bwd(x, w, target, lse, dlogp)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    l2, e2 = jet.head_logp(x, w, target, stream=side)
    dx2, dw2 = jet.head_logp_bwd(x, w, target, e2, dlogp, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in ((logp, l2), (lse, e2), (dx, dx2), (dw, dw2)))
    out = [torch.zeros_like(t) for t in (logp, lse, dx, dw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        jet.jet_head_logp(x, w, target, 1.0, out[0], out[1])
        jet.jet_head_logp_bwd(x, w, target, out[1], dlogp, 1.0, out[2], out[3])
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, (logp, lse, dx, dw)))
    code, word = jet.device_status()
    assert code == 0, hex(word)


def test_refusals(jet):
    x, w, target, dlogp = make(4, 64, 50, 11)
    with pytest.raises(ValueError):
        jet.head_logp(x, w[:, :56].contiguous(), target)
    with pytest.raises(ValueError):
        jet.head_logp(x.t(), w, target)
    with pytest.raises(TypeError):
        jet.head_logp(x, w, target.int())
    with pytest.raises(TypeError):
        jet.head_logp(x.float(), w, target)
    with pytest.raises(jet.JetError):
        jet.head_logp(x, w, target, scale=0.0)
