"""The workspace of the head's backward over its range of sizes; CPU only."""
import pytest

from fp8_block_quantized_gb300 import binding


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 128, 129, 1000, 4096, 65536])
@pytest.mark.parametrize("V", [1, 1000, 151937, 2000003, (1 << 24) - 1])
@pytest.mark.parametrize("K", [8, 4096])
def test_gradients_of_the_logits_take_half_a_gigabyte(T, V, K):
    """The workspace is d of a piece, dx of its ranges (512 MB, or one range of both parts) and dx
    so far, each up to a multiple of 256 bytes."""
    got = binding.load().jet_workspace_bytes(binding.OP["head_logp_bwd"], T, V, K)
    rows = 2 * -(-T // 64) * 64 if T <= 128 else T
    d = max(512 << 20, 2 * rows * 4096)
    assert 0 < got <= d + max(512 << 20, 4 * rows * K) + 4 * T * K + 3 * 256
