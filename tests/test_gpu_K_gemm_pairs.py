"""GPU test of the products by CTA pairs in short calls, each call's first tiles
behind the last's."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1024, 256, 128), (1152, 512, 256), (2048, 128, 512)])
def test_short_products_one_behind_another(torch_cuda, M, N, K):
    import fp8_block_quantized_gb300 as jet
    g = torch.Generator(device="cuda").manual_seed(M)
    x, w = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in ((M, K), (N, K)))
    qx, sx = jet.quant_act_1x128(x)
    qw, sw = jet.quant_w_128x128(w)
    y = jet.gemm_fp8_fwd(qx, sx, qw, sw)
    for _ in range(50):
        again = jet.gemm_fp8_fwd(qx, sx, qw, sw)
    torch.cuda.synchronize()
    code, word = jet.device_status()
    assert code == 0, hex(word)
    assert torch.equal(y, again)
    # E4M3 operands are off by 2^-4 of themselves each, the output by 2^-8; sums in binary32
    size = x.double().abs() @ w.double().abs().t()
    assert ((y.double() - x.double() @ w.double().t()).abs() <= (2.0 ** -3 + 2.0 ** -8 + 2.0 ** -7) * size).all()
