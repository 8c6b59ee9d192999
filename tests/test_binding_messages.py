"""A refused tensor's message names that tensor and how many dimensions it has; CPU only."""
import pytest
import torch

import fp8_block_quantized_gb300 as jet

BF16 = torch.bfloat16


def test_dimensions():
    f, pos = torch.empty((32,), dtype=torch.float64), torch.empty((4,), dtype=torch.int64)
    flat, q = torch.empty((4, 64), dtype=BF16), torch.empty((4, 2, 64), dtype=BF16)
    scale, cache = torch.empty((2,)), torch.empty((4, 2, 64), dtype=torch.uint8)
    with pytest.raises(ValueError, match=r"^k: expected three dimensions, got 2$"):
        jet.jet_rope(None, flat, f, pos, None, flat)
    with pytest.raises(ValueError, match=r"^q: expected three dimensions, got 2$"):
        jet.jet_rope(flat, None, f, pos, flat, None)
    with pytest.raises(ValueError, match=r"^q: expected three dimensions, got 2$"):
        jet.jet_rope_kv_cache_write(flat, q, q, f, pos, scale, scale, pos, flat, cache, cache)
    with pytest.raises(ValueError, match=r"^logits: expected two dimensions, got 3$"):
        jet.jet_sample(q, scale, None, None, None, None, pos, scale, scale, pos)
