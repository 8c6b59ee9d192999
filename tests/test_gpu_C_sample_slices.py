"""GPU tests of sampling from slices of a batch, whose first logit lies at any
element, and the argument checks of that form."""
import ctypes

import pytest
import torch

from fp8_block_quantized_gb300 import binding
from tests.test_gpu_9_sample import logits, run

OK, NULL, SHAPE, ALIGN = range(4)


@pytest.fixture(scope="module")
def jet(torch_cuda):
    import fp8_block_quantized_gb300 as j
    j.load()
    return j


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,V,ld", [(9, 5, 5), (9, 4099, 4099), (9, 32001, 32003), (3, 50257, 50257),
                                    (320, 1001, 1001)])
@pytest.mark.parametrize("filters", [False, True])
def test_slices_of_a_batch(jet, dtype, B, V, ld, filters):
    """The rows from each of the first eight on, and columns cut in front: the
    definition's tokens, and the same bits as from an aligned copy."""
    x, u = logits(B, V, B + V, dtype, ld)
    kw = dict(k=torch.full((B,), 40), p=torch.full((B,), 0.9)) if filters else {}
    for row in range(min(8, B)):
        for col in (0, 1, 2):
            part = {n: t[row:] for n, t in kw.items()}
            got = run(jet, x[row:, col:], u[row:], **part)
            want = run(jet, x[row:, col:].contiguous().clone(), u[row:], **part)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (row, col)


def test_refusals():
    lib = binding.load()
    P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(10)]    # aligned, never dereferenced

    def call(at, dtype=0, B=4, V=1000, u=P[1]):
        return lib.jet_sample_unaligned(ctypes.c_void_p(at), dtype, B, V, 1000, u, None, None, None, None,
                                        P[6], P[7], P[8], P[9], None)
    assert call(0x10001) == ALIGN and call(0x10002, dtype=1) == ALIGN and call(0x10001, u=None) == NULL
    assert call(0x10002, V=1001) == SHAPE and call(0x10002, B=-1) == SHAPE
    if not torch.cuda.is_available():                              # else they would be launched
        assert call(0x10002) == call(0x10004, dtype=1) == call(0x10000) == 5
