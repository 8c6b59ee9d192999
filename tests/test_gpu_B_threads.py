"""GPU tests of calls from several host threads: one thread's sizes do not
change what another's launch may have."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
CALLS = 3000


@pytest.fixture(scope="module")
def jet(torch_cuda):
    import fp8_block_quantized_gb300 as j
    j.load()
    return j


def together(*calls):
    """Each call CALLS times in a thread of its own, on a stream of its own."""
    torch.cuda.synchronize()
    start, errors = threading.Barrier(len(calls)), []

    def work(call):
        stream = torch.cuda.Stream()
        start.wait()
        try:
            for _ in range(CALLS):
                call(stream)
        except Exception as e:
            errors.append(e)
        stream.synchronize()
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_sampling_of_short_and_long_rows(jet):
    """Both with filters, so that the slices of the rows lie in shared memory."""
    def caller(V):
        x = torch.randn((1, V), generator=torch.Generator().manual_seed(V)).cuda()
        u, k = torch.full((1,), 0.4, device="cuda"), torch.full((1,), 20, dtype=torch.int32, device="cuda")
        want = jet.sample(x, u, top_k=k)
        out = [torch.empty_like(t) for t in want]
        return lambda s: jet.jet_sample(x, u, None, k, None, None, *out, stream=s), want, out
    calls, wants, outs = zip(*map(caller, (4000, 262144, 70000)))
    together(*calls)
    torch.cuda.synchronize()
    for want, out in zip(wants, outs):
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_norms_of_long_rows(jet):
    """Rows that need more shared memory than every launch may have, of lengths
    that go to one kernel."""
    def forward(K):
        x, g = torch.randn((2, K), device="cuda").to(BF16), torch.ones((K,), dtype=BF16, device="cuda")
        want = jet.add_rmsnorm_quant_1x128(x, x, g, with_rstd=True)
        out = [torch.empty_like(t) for t in want]
        return lambda s: jet.jet_add_rmsnorm_quant_1x128(x, x, g, 1e-5, *out, stream=s), want, out
    calls, wants, outs = zip(*map(forward, (20736, 24576, 32768)))
    together(*calls)
    torch.cuda.synchronize()
    for want, out in zip(wants, outs):
        assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("sizes", [((4096, 1), (4096, 3), (3584, 2)), ((8192, 1), (8192, 3), (7168, 2)),
                                   ((10240, 1), (16384, 3), (12288, 2)), ((20480, 1), (28672, 2), (18432, 3))])
def test_norm_gradients(jet, sizes):
    """Rows and numbers of gradients that go to one kernel with other needs."""
    def backward(K, n):
        x, g = torch.randn((2, K), device="cuda").to(BF16), torch.ones((K,), dtype=BF16, device="cuda")
        rstd, ws = torch.ones((2,), device="cuda"), torch.empty((2 * K * 4,), dtype=torch.uint8, device="cuda")
        want = jet.add_rmsnorm_bwd(x, g, rstd, [x] * n)
        out = [torch.empty_like(t) for t in want]
        return lambda s: jet.jet_add_rmsnorm_bwd(x, g, rstd, [x] * n, None, *out, ws, stream=s), want, out
    calls, wants, outs = zip(*(backward(*s) for s in sizes))
    together(*calls)
    torch.cuda.synchronize()
    for want, out in zip(wants, outs):
        assert all(torch.equal(a, b) for a, b in zip(want, out))
