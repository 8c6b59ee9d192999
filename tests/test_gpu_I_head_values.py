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
