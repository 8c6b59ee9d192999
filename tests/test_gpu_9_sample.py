"""GPU tests of the sampler against its definition written out per row in 64
bits (the binary32 differences, products and weights of the definition
aside).  The weights may differ by an ulp of e^z between the two, so a drawn token is
accepted when u S lies within that of its interval."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# expf within 2 ulps: every running sum within 2^-22 of itself; a little more for the quotients
SLACK = 2.0 ** -21


@pytest.fixture(scope="module")
def jet(torch_cuda):
    import fp8_block_quantized_gb300 as j
    j.load()
    return j


def weights(x, T):
    x = np.where(np.isnan(x), -np.inf, x).astype(np.float32)
    m = x.max()
    inv = np.float32(1.0) / np.float32(T if T > 0 else 1.0)
    with np.errstate(all="ignore"):
        z = np.where(x == m, np.float32(0), (x - m).astype(np.float32) * inv).astype(np.float32)
    return x, np.where(x == -np.inf, 0.0, np.exp(z.astype(np.float64)).astype(np.float32)).astype(np.float64)


def check_row(x, u, T, k, p, mp, token, logp, logp_all, kept):
    x, w = weights(x, T)
    if x.max() == -np.inf:
        assert token == -1 and kept == 0 and np.isnan(logp) and np.isnan(logp_all)
        return
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    k = 1 if T <= 0 else k if k > 0 else len(order)
    order = order[:k]
    before = np.concatenate([[0.0], np.cumsum(w[order])])
    n_lo = n_hi = len(order)
    if p < 1:
        target = max(p, 0.0) * before[-1]
        n_lo = max(1, int((before[:-1] < target * (1 - SLACK)).sum()))
        n_hi = max(1, int((before[:-1] < target * (1 + SLACK)).sum()))
    if mp > 0:
        ok = lambda n, s: max(1, int((w[order[:n]] >= np.float32(min(mp, 1.0)) * s).sum()))
        n_lo, n_hi = ok(n_lo, 1 + 2.0 ** -22), ok(n_hi, 1 - 2.0 ** -22)
    assert n_lo <= kept <= n_hi, (kept, n_lo, n_hi)
    idx = np.sort(order[:kept])
    at = np.searchsorted(idx, token)
    assert at < len(idx) and idx[at] == token, "a token that was not kept"
    cum = np.cumsum(w[idx])
    S = cum[-1]
    lo = cum[at - 1] if at else 0.0
    assert lo - SLACK * S <= u * S <= cum[at] + SLACK * S, (lo / S, u, cum[at] / S)
    for got, total in ((logp, S), (logp_all, w.sum())):
        ref = np.log(w[token] / total)
        assert abs(got - ref) <= 2.0 ** -20 + 2.0 ** -22 * abs(ref), (got, ref)


def run(jet, x, u, T=None, k=None, p=None, mp=None):
    dev = lambda v, t: None if v is None else torch.as_tensor(v).to(t).cuda()
    out = jet.sample(x, dev(u, F32), dev(T, F32), dev(k, torch.int32), dev(p, F32), dev(mp, F32))
    torch.cuda.synchronize()
    B = x.shape[0]
    xs = x.float().cpu().numpy()
    full = lambda v, d: np.full(B, d) if v is None else torch.as_tensor(v).numpy()
    rows = zip(xs, torch.as_tensor(u).to(F32).double().numpy(), full(T, 1.0), full(k, 0), full(p, 1.0), full(mp, 0.0),
               *(t.cpu().numpy() for t in out))
    for r in rows:
        check_row(*r)
    return out


def logits(B, V, seed, dtype=F32, ld=None, std=2.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, ld or V), generator=g) * std
    x[:, :V].scatter_add_(1, torch.randint(0, V, (B, min(V, 24)), generator=g),
                          4 * torch.rand((B, min(V, 24)), generator=g) + 2)
    return x.to(dtype).cuda()[:, :V], torch.rand((B,), generator=g)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,V,ld", [(1, 1, 1), (3, 2, 2), (2, 31, 40), (5, 100, 100), (1, 50257, 50257),
                                    (4, 32000, 32000), (40, 4099, 4101), (3, 128256, 128256),
                                    (160, 1000, 1003), (2, 151937, 151937), (1, 262144, 262144),
                                    (30, 128256, 128264)])
def test_whole_distribution(jet, dtype, B, V, ld):
    x, u = logits(B, V, B + V, dtype, ld)
    run(jet, x, u)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [7, 1000, 32003, 128256])
@pytest.mark.parametrize("kind", ["temperature", "top_k", "top_p", "min_p", "all"])
def test_filters(jet, dtype, V, kind):
    B = 12
    x, u = logits(B, V, V, dtype)
    r = torch.arange(B)
    pick = lambda v: torch.tensor(v)[r % len(v)]
    kw = {}
    if kind in ("temperature", "all"):
        kw["T"] = pick([1.0, 0.6, 0.0, 1.7, 0.05, -1.0, 30.0])
    if kind in ("top_k", "all"):
        kw["k"] = pick([1, 2, 50, 1000, 0, -3, V, V - 1, 20000, 10 ** 9])
    if kind in ("top_p", "all"):
        kw["p"] = pick([0.9, 0.5, 1.0, 0.999, 0.0, 0.05, 2.0, -1.0])
    if kind in ("min_p", "all"):
        kw["mp"] = pick([0.0, 0.1, 0.001, 1.0, 3.0, -1.0])
    run(jet, x, u, **kw)


def test_masked_and_odd_values(jet):
    x, u = logits(10, 5000, 1)
    inf = float("inf")
    x[0] = -inf
    x[1] = float("nan")
    x[2, :4990] = -inf
    x[3, 1::2] = float("nan")
    x[4, 77] = inf
    x[5, [3, 4000]] = inf
    x[6] = torch.finfo(F32).min
    x[7] = 0.0
    x[7, ::2] = -0.0
    x[8] = torch.finfo(F32).min
    x[8, 1234] = 0.0
    x[9] = 1e-40
    T = torch.tensor([1.0, 0.5, 0.7, 1.0, 1.0, 2.0, 1.0, 1.0, 1.0, 1.0])
    a = run(jet, x, u, T)
    run(jet, x, u)
    run(jet, x, u, T, k=torch.full((10,), 6), p=torch.full((10,), 0.7))
    run(jet, x, u, T, k=torch.full((10,), 4000), p=torch.full((10,), 0.93), mp=torch.full((10,), 0.5))
    assert int(a[0][4]) == 77 and int(a[0][5]) in (3, 4000) and int(a[0][8]) == 1234
    g = run(jet, x, u, torch.zeros(10))
    assert g[0].tolist()[5:9] == [3, 0, 0, 1234]            # greedy: the lowest index of the largest


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,V", [(3, 5), (6, 4097), (6, 128256), (400, 33001)])
def test_a_few_odd_values(jet, dtype, B, V):
    """Single NaN and infinities at a row's ends and inside: the threads that read
    them and those that do not draw from the same weights."""
    x, u = logits(B, V, 17)
    x = x.to(dtype)
    i = torch.arange(B)
    x[i, (i * 7919) % V] = float("nan")
    x[::3, 0] = float("nan")
    x[1::3, V - 1] = float("nan")
    x[2::3, V // 2] = -float("inf")
    x[B - 1, V // 3] = float("inf")
    run(jet, x, u)
    run(jet, x, u, p=torch.full((B,), 0.9))


@pytest.mark.parametrize("n", [2047, 2048, 2049, 4095, 4096, 6000])
def test_as_many_candidates_as_the_list_takes(jet, n):
    """n logits far above the others, one or several of them a thread."""
    x = torch.full((8, 128256), -20.0, device="cuda")
    for b, step in enumerate((1, 3, 8, 19, 21, 4, 16, 2)):
        x[b, torch.arange(n) * step + 5 * b] = torch.linspace(0.0, 0.2, n, device="cuda")
    u = torch.linspace(0.0, 0.999, 8)
    run(jet, x, u, p=torch.tensor([0.1, 0.5, 0.9, 0.99, 0.999, 0.3, 0.7, 0.95]))
    run(jet, x, u, mp=torch.full((8,), 0.5))
    run(jet, x, u, k=torch.tensor([n - 1, n, n + 1, 5, 2048, 2049, 1000, n // 2]), p=torch.full((8,), 0.9))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [600, 40000, 128256])
def test_ties(jet, dtype, V):
    """Equal logits are kept by rising index, in numbers that no ranking list holds."""
    B = 8
    x = torch.zeros((B, V), dtype=dtype, device="cuda")
    x[4:, 5::3] = 1.0
    x[6:, 7::11] = 1.0
    u = torch.tensor([0.0, 0.25, 0.5, 0.999, 0.1, 0.3, 0.6, 0.99])
    run(jet, x, u)
    run(jet, x, u, k=torch.tensor([1, 2, 513, V - 1, 100, V // 2, V // 3 + 1, 550]))
    run(jet, x, u, p=torch.tensor([0.5, 0.25, 0.001, 0.999, 0.3, 0.9, 0.5, 0.7]))
    t = run(jet, x, u, k=torch.full((B,), 1))
    assert t[0].tolist()[:4] == [0] * 4


@pytest.mark.parametrize("T", [0.01, 1.0, 100.0, 1e6])
def test_narrow_and_wide_spreads(jet, T):
    """Steps of z that hold far more tokens than are ranked at once, and filters
    whose cut lies among weights that round to nothing."""
    x, u = logits(6, 100000, 3)
    t = torch.full((6,), T)
    run(jet, x, u, t, k=torch.tensor([5, 700, 30000, 99999, 60000, 1]))
    run(jet, x, u, t, p=torch.tensor([0.1, 0.5, 0.9, 0.99, 0.9999, 0.3]))
    run(jet, x, u, t, k=torch.tensor([600, 5000, 80000, 99998, 3, 100]),
        p=torch.tensor([0.1, 0.5, 0.9, 0.99, 0.9999, 0.3]))


def test_the_batch_does_not_change_a_row(jet):
    """One row alone (eight CTAs a row), in a middle and in a large batch (fewer
    CTAs a row): the same token and log-probability bits."""
    V = 32000
    x, u = logits(300, V, 11)
    T, p = torch.full((300,), 0.8), torch.full((300,), 0.95)
    big = run(jet, x, u, T, p=p)
    for lo, hi in ((7, 8), (100, 120), (290, 300)):
        for n in (lo,) if hi - lo == 1 else range(lo, hi, 4):
            part = jet.sample(x[n:n + 1].clone(), u[n:n + 1].cuda(), T[:1].cuda(), None, p[:1].cuda())
            for a, b in zip(part, big):
                assert torch.equal(a, b[n:n + 1])


@pytest.mark.parametrize("B", [40, 120, 153, 185, 200, 310, 700, 1300])
@pytest.mark.parametrize("V,dtype", [(700, F32), (4099, F32), (32000, BF16), (50257, F32), (128256, BF16), (151937, F32)])
def test_any_number_of_rows_without_filters(jet, B, V, dtype):
    """Every split of rows into CTAs: every 29th row as if alone."""
    if B * V > 4e7:
        B = max(40, int(4e7) // V)
    g = torch.Generator(device="cuda").manual_seed(B + V)
    x = (torch.randn((B, V), generator=g, device="cuda") * 2.5).to(dtype)
    u = torch.rand((B,), generator=g, device="cuda")
    full = jet.sample(x, u)
    for i in range(0, B, 29):
        one = jet.sample(x[i:i + 1].clone(), u[i:i + 1].clone())
        for a, b in zip(one, full):
            assert torch.equal(a, b[i:i + 1]), (i, a, b[i])


@pytest.mark.parametrize("B", [17, 20, 26, 33, 60, 75, 100, 150, 300])
@pytest.mark.parametrize("V,dtype", [(33001, F32), (128256, BF16), (151937, F32), (262144, BF16), (262143, F32)])
def test_any_number_of_rows_gives_a_row_the_same(jet, B, V, dtype):
    """Clusters of every size, one and two CTAs an SM: every 7th row as if alone."""
    g = torch.Generator(device="cuda").manual_seed(B + V)
    x = (torch.randn((B, V), generator=g, device="cuda") * 2.5).to(dtype)
    u = torch.rand((B,), generator=g, device="cuda")
    r = torch.arange(B, device="cuda")
    pick = lambda v, t: torch.tensor(v, device="cuda", dtype=t)[r % len(v)]
    T, k = pick([1.0, 0.6, 0.0, 1.7, 0.9], F32), pick([0, 50, 3000, V // 2], torch.int32)
    p, mp = pick([0.95, 1.0, 0.5], F32), pick([0.0, 0.01], F32)
    for f in ((T, k, p, mp), (None, None, p, None), (None, k, None, None)):
        full = jet.sample(x, u, *f)
        for i in range(0, B, 7):
            one = jet.sample(x[i:i + 1].clone(), u[i:i + 1], *(None if v is None else v[i:i + 1] for v in f))
            for a, b in zip(one, full):
                assert torch.equal(a, b[i:i + 1]), (i, a, b[i])


def test_frequencies_of_an_even_grid(jet):
    """u on a grid of n points draws every token n p times, up to one."""
    n, V = 4096, 300
    g = torch.Generator().manual_seed(5)
    row = torch.randn((V,), generator=g) * 2
    x = row.expand(n, V).contiguous().cuda()
    token, *_ = jet.sample(x, ((torch.arange(n) + 0.5) / n).cuda(), top_k=torch.full((n,), 40, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    count = torch.bincount(token.cpu(), minlength=V).double()
    top = row.topk(40).indices
    p = torch.zeros(V, dtype=torch.float64)
    p[top] = torch.softmax(row[top].double(), 0)
    assert ((count - n * p).abs() <= 1 + n * 2.0 ** -20).all()


def test_odd_uniform_numbers(jet):
    x, _ = logits(6, 500, 2)
    x[:, 0] = -float("inf")
    out = jet.sample(x, torch.tensor([1.0, 2.0, -0.5, float("nan"), 0.0, 0.9999999]).cuda())
    torch.cuda.synchronize()
    tok = out[0].tolist()
    assert all(1 <= t < 500 for t in tok)
    assert tok[2] == tok[3] == tok[4] == 1


def test_empty_batch(jet):
    out = jet.sample(torch.empty((0, 100), device="cuda"), torch.empty((0,), device="cuda"))
    torch.cuda.synchronize()
    assert out[0].shape == (0,)


@pytest.mark.parametrize("gap", [0.3, 0.45, 1.7])
def test_many_long_flat_rows(jet, gap):
    """Hundreds of long rows (one CTA a row, hundreds of logits a thread) of two
    levels, whose weights all carry large low-order parts: the same tokens and
    log-probabilities as each row alone, and the sums of the definition."""
    B, V = 310, 190001
    x = torch.zeros((1, V), dtype=BF16, device="cuda")
    x[0, 1:] = -gap
    x = x.expand(B, V).contiguous()
    u = (torch.arange(B) + 0.5) / B
    out = jet.sample(x, u.cuda())
    alone = jet.sample(x[7:8].clone(), u[7:8].cuda())
    torch.cuda.synchronize()
    for a, b in zip(out, alone):
        assert torch.equal(a[7:8], b)
    xs = x[0].float().cpu().numpy()
    for b in (0, 1, 150, 309):
        check_row(xs, float(u[b]), 1.0, 0, 1.0, 0.0, *(t[b].item() for t in out))
