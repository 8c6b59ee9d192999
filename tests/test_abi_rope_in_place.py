"""Rotary positions in place need the input's strides for the output: another
stride would have tokens written before they are read.  CPU only."""
import ctypes

import pytest
import torch

from fp8_block_quantized_gb300 import binding

OK, NULL, SHAPE, ALIGN, CUDA, DEVICE = range(6)
P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(12)]   # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; valid arguments would be launched")
    return binding.load()


def rope(lib, T=10, q=P[0], ldq=512, qo=P[4], ldqo=512, k=P[1], ldk=256, ko=P[5], ldko=256):
    return lib.jet_rope(q, ldq, 4, k, ldk, 2, T, 128, 64, P[2], P[3], 0, 1.0, 0, qo, ldqo, ko, ldko, None)


def test_rope(lib):
    assert rope(lib) == DEVICE
    assert rope(lib, qo=P[0], ko=P[1]) == DEVICE
    assert rope(lib, ldqo=1024, ldko=512) == DEVICE                 # not in place
    assert rope(lib, qo=P[0], ldqo=1024) == SHAPE
    assert rope(lib, qo=P[0], ldq=520) == SHAPE
    assert rope(lib, ko=P[1], ldko=264) == SHAPE
    assert rope(lib, qo=P[0], ldqo=1024, T=1) == DEVICE             # one token has no stride


def test_rope_with_the_cache_write(lib):
    def write(qo, ldqo, T=10):
        return lib.jet_rope_kv_cache_write(P[0], 512, 4, P[1], 256, P[2], 256, 2, T, 128, 64, P[3], P[4], 0, 1.0,
                                           P[5], P[6], P[7], qo, ldqo, P[9], P[10], 64, None)
    assert write(P[8], 1024) == write(P[0], 512) == write(P[0], 1024, 1) == DEVICE
    assert write(P[0], 1024) == SHAPE
