"""GPU tests of the head's log-probabilities and gradients: CTA pairs with little
to do, targets whose probability is near one, many products a logit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def jet(torch_cuda):
    import fp8_block_quantized_gb300 as j
    j.load()
    return j


def make(T, K, V, seed, std=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, K), generator=g, device="cuda").to(BF16)
    w = (torch.randn((V, K), generator=g, device="cuda") * std * K ** -0.5).to(BF16)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    return x, w, target, torch.randn((T,), generator=g, device="cuda")


@pytest.mark.parametrize("T,K,V", [(257, 64, 100), (257, 1024, 5000), (384, 512, 129), (640, 64, 20000)])
def test_short_calls_one_behind_another(jet, T, K, V):
    """Products by CTA pairs of which the second has rows in only some tiles or none, each call's
    first ones behind the last's."""
    x, w, target, dlogp = make(T, K, V, T + V)
    logp, lse = jet.head_logp(x, w, target)
    dx, dw = jet.head_logp_bwd(x, w, target, lse, dlogp)
    for _ in range(30):
        l2, e2 = jet.head_logp(x, w, target)
        dx2, dw2 = jet.head_logp_bwd(x, w, target, e2, dlogp)
    torch.cuda.synchronize()
    code, word = jet.device_status()
    assert code == 0, hex(word)
    assert all(torch.equal(a, b) for a, b in ((logp, l2), (lse, e2), (dx, dx2), (dw, dw2)))


def test_a_short_last_piece(jet):
    """So many tokens that the vocabulary is walked in pieces of 4096, of which 100 are left."""
    T, K, V, v0 = 66001, 64, 19 * 4096 + 100, 19 * 4096
    x, w, target, dlogp = make(T, K, V, 1)
    target[::3] = v0 + target[::3] % 100
    _, lse = jet.head_logp(x, w, target)
    dw = torch.full_like(w, 7.0)
    jet.jet_head_logp_bwd(x, w, target, lse, dlogp, 1.0, None, dw)
    z = x.double() @ w[v0:].double().t()
    p = torch.exp(z - lse.double()[:, None])
    hot = (target[:, None] == torch.arange(v0, V, device="cuda")).double()
    d = dlogp.double()[:, None] * (hot - p)
    # a logit: sums of 16 products into binary32 (2^-22 each of what was added up), lse's rounding and the
    # argument's; d to BF16; sums of T terms; the output's rounding
    size = x.double().abs() @ w[v0:].double().abs().t()
    off = dlogp.double().abs()[:, None] * p * (size * (K / 16 + 2) * 2.0 ** -22 + (z.abs() + lse.double().abs()[:, None] + 8) * 2.0 ** -22)
    off += 2.0 ** -8 * d.abs()
    ref = d.t() @ x.double()
    bound = off.t() @ x.double().abs() + 2.0 ** -8 * ref.abs() + (T / 16 + 20) * 2.0 ** -22 * (d.abs().t() @ x.double().abs())
    assert ((dw[v0:].double() - ref).abs() <= bound).all()
    assert not (dw == 7.0).all(1).any()


@pytest.mark.parametrize("T", [32, 200])
@pytest.mark.parametrize("K", [4096, 16384])
def test_gradients_of_confident_tokens(jet, T, K):
    """Logits of 20 to 100 whose products all have one sign; the target's probability is about 0.95.
    Against the gradient by the formula, not by the lse that the forward gave."""
    V = 600
    x, w, target, _ = make(T, K, V, K + T, std=0.1)
    target = torch.randperm(V // 2, device="cuda")[:T]
    z = torch.linspace(20, 100, T, device="cuda")
    unit = x.float() / x.float().square().sum(1, keepdim=True)
    w[target] = (unit * z[:, None]).to(BF16)
    w[target + V // 2] = (unit * (z - 3)[:, None]).to(BF16)
    dlogp = torch.where(torch.arange(T, device="cuda") % 2 == 0, 1.0, -0.5)
    _, lse = jet.head_logp(x, w, target)
    dx, dw = jet.head_logp_bwd(x, w, target, lse, dlogp)
    x64, w64 = x.double(), w.double()
    z64 = x64 @ w64.t()
    p = torch.softmax(z64, 1)
    hot = torch.zeros_like(p).scatter_(1, target[:, None], 1.0)
    up = dlogp.double()[:, None]
    d = up * (hot - p)
    at = torch.arange(T, device="cuda")
    assert (d[at, target].abs() < 0.1 * up.abs()[:, 0]).all()
    # a logit: 64 sums of 16 products at a time into binary32, each off by a unit of 2^-22 of what was added up,
    # then the chunks'; alike in both calls, so that a probability is off by p (1 - p) times two of that;
    # and the roundings of lse, of its product and the exponential's argument
    dz = (x64.abs() @ w64.abs().t()).amax(1, keepdim=True) * (66 + K / 1024) * 2.0 ** -22
    top = z64.abs().amax(1, keepdim=True)
    off = up.abs() * p * ((1 - p) * 2 * dz + (2 * top + 8) * 2.0 ** -22) + 2.0 ** (-16 if T <= 128 else -8) * d.abs()
    for got, ref, bound, mag, n in ((dx, d @ w64, off @ w64.abs(), d.abs() @ w64.abs(), V),
                                    (dw, d.t() @ x64, off.t() @ x64.abs(), d.abs().t() @ x64.abs(), T)):
        bound = bound + 2.0 ** -8 * ref.abs() + mag * (n / 16 + 20) * 2.0 ** -22 + 1e-38
        assert ((got.double() - ref).abs() <= bound).all(), ((got.double() - ref).abs() / bound).max()


def test_few_tokens_of_a_vocabulary_in_pieces(jet):
    """Up to 128 tokens, whose d has two parts: pieces of the vocabulary and dx added up over them."""
    T, K, V = 3, 64, 2200000
    x, w, target, dlogp = make(T, K, V, 2)
    target[0] = V - 1
    _, lse = jet.head_logp(x, w, target)
    dx, dw = jet.head_logp_bwd(x, w, target, lse, dlogp)
    x64, w64 = x.double(), w.double()
    z = x64 @ w64.t()
    p = torch.exp(z - lse.double()[:, None])
    up = dlogp.double()[:, None]
    d = (-up * p).scatter_add_(1, target[:, None], up)
    # a logit: sums of 16 products into binary32; lse's rounding and the argument's; d in two parts; sums of V or
    # T terms, the outputs' rounding
    dz = (x64.abs() @ w64.abs().t()) * (K / 16 + 2) * 2.0 ** -22
    off = up.abs() * p * (2 * dz + (z.abs() + lse.double().abs()[:, None] + 8) * 2.0 ** -22) + 2.0 ** -16 * d.abs()
    for got, ref, bound, mag, n in ((dx, d @ w64, off @ w64.abs(), d.abs() @ w64.abs(), V),
                                    (dw, d.t() @ x64, off.t() @ x64.abs(), d.abs().t() @ x64.abs(), T)):
        bound = bound + 2.0 ** -8 * ref.abs() + mag * (n / 16 + 20) * 2.0 ** -22 + 1e-38
        assert ((got.double() - ref).abs() <= bound).all()
