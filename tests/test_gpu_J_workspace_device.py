"""GPU tests of workspaces given to the attention and the head: what another device
owns is refused.  One GPU is enough: the workspace is a tensor without memory."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jet(torch_cuda):
    import fp8_block_quantized_gb300 as j
    j.load()
    return j


class NoMemory(torch.Tensor):
    @staticmethod
    def __new__(cls, n, device):
        return torch.Tensor._make_wrapper_subclass(cls, (n,), dtype=torch.uint8, device=device)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(func)


@pytest.fixture(scope="module")
def elsewhere(torch_cuda):
    return NoMemory(1 << 24, "cuda:1")


def test_head(jet, elsewhere):
    x, w = (torch.ones((n, 64), dtype=torch.bfloat16, device="cuda") for n in (4, 50))
    t = torch.zeros((4,), dtype=torch.int64, device="cuda")
    logp, lse = torch.ones((4,), device="cuda"), torch.ones((4,), device="cuda")
    with pytest.raises(ValueError, match="current device"):
        jet.jet_head_logp(x, w, t, 1.0, logp, lse, ws=elsewhere)
    with pytest.raises(ValueError, match="current device"):
        jet.jet_head_logp_bwd(x, w, t, lse, logp, 1.0, torch.empty_like(x), torch.empty_like(w), ws=elsewhere)
    assert (logp == 1).all() and (lse == 1).all()


def test_attention(jet, elsewhere):
    z = lambda *s, d: torch.zeros(s, dtype=d, device="cuda")
    q, cache, one = z(1, 4, 64, d=torch.bfloat16), z(16, 1, 64, d=torch.uint8), z(1, d=torch.float32)
    off = torch.tensor([0, 1], device="cuda")
    with pytest.raises(ValueError, match="current device"):
        jet.jet_kv_attention(q, cache, cache, one, one, z(1, 1, d=torch.int32), 16, off, z(1, d=torch.int32),
                             torch.empty_like(q), ws=elsewhere)
