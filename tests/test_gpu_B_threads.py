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
