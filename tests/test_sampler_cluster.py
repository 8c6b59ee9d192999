"""The sampler's cluster protocol, on the CPU: the kernel's own source is run
with every thread a fiber (tests/cluster/), under schedules in which one CTA of
the cluster falls behind the others from a given cluster barrier on.  Every
schedule has to end, and to give what the definition gives."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from tests.test_gpu_9_sample import check_row

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(os.path.dirname(HERE), "fp8_block_quantized_gb300", "csrc", "sample.cu")


@pytest.fixture(scope="module")
def emulated(tmp_path_factory):
    out = tmp_path_factory.mktemp("cluster")
    text = open(SOURCE).read()
    text = text[text.index("namespace {"):text.index("template <int kBytes>\nbool aligned_to")] + "\n}\n"

    def replace(pattern, by):
        nonlocal text
        text, n = re.subn(pattern, by, text, flags=re.S)
        assert n, pattern
    # the copies to shared memory happen at once here, so there is nothing to wait for
    replace(r'asm volatile\("cp\.async\.cg.*?"memory"\);', "memcpy(dst, src, 16);")
    replace(r'asm volatile\("cp\.async\.(wait|commit)_group.*?"memory"\);', ";")
    replace(r"extern __shared__ [^;]* smem\[\];", "unsigned char *smem = emu::smem();")
    assert "asm" not in text
    (out / "sample_source.inc").write_text(text)
    lib = out / "sampler.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-U_FORTIFY_SOURCE", "-ffp-contract=off",
                    "-Wno-narrowing", "-I", str(out), "-I", os.path.join(HERE, "cluster"),
                    os.path.join(HERE, "cluster", "sampler.cpp"), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


def sample(lib, x, C, u, T, k, p, mp, lag, who, start):
    """(status, early accesses, cluster barriers, outputs) of one row."""
    arr = lambda v, t: None if v is None else np.array([v], t)
    ptr = lambda a: None if a is None else ctypes.c_void_p(a.ctypes.data)
    ins = [arr(u, np.float32), arr(T, np.float32), arr(k, np.int32), arr(p, np.float32), arr(mp, np.float32)]
    outs = [np.zeros(1, np.int64), np.zeros(1, np.float32), np.zeros(1, np.float32), np.zeros(1, np.int32)]
    early, syncs = ctypes.c_int(0), ctypes.c_int(0)
    st = lib.sample_row(ctypes.c_void_p(x.data_ptr()), int(x.dtype == torch.bfloat16), x.numel(), C,
                        *map(ptr, ins), lag, who, start, *map(ptr, outs), ctypes.byref(early), ctypes.byref(syncs))
    return st, early.value, syncs.value, [o[0] for o in outs]


def row(V, dtype, seed, std=2.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((V,), generator=g) * std
    x[torch.randint(0, V, (12,), generator=g)] += 5.0
    x[torch.randint(0, V, (max(1, V // 50),), generator=g)] = -float("inf")
    return x.to(dtype)


# every way through the kernel: (settings T, k, p, min-p; spread of the logits)
WAYS = {
    "plain": ((None, None, None, None), 2.5),
    "temperature": ((0.7, None, None, None), 2.5),
    "greedy": ((0.0, None, None, None), 2.5),
    "one": ((1.0, 1, None, None), 2.5),
    "first": ((1.0, None, 0.0, None), 2.5),
    "short list": ((1.0, 20, 0.9, None), 2.5),
    "long list": ((1.0, 900, 0.95, 0.001), 2.5),
    "min-p of a flat row": ((1.0, None, None, 0.5), 0.01),
    "nucleus of a flat row": ((1.0, None, 0.9, None), 0.01),
    "top-k of a flat row": ((1.0, 3500, None, None), 0.001),
    "both of a flat row": ((1.0, 3500, 0.8, 0.2), 0.01),
}


NOBODY, CTA, OTHERS, WARP = range(4)
V, C, U = 6001, 3, 0.37


def check_schedules(lib, way, dtype, lags, starts, early=True):
    """(lag, who) falling behind from each of the barriers `starts` on: every
    thread ends, the outputs are the definition's, and no CTA that is not there
    is touched, where that is asked for."""
    (T, k, p, mp), std = WAYS[way]
    x = row(V, dtype, 3, std)
    full = lambda v, d: d if v is None else v

    def check(*schedule):
        status, n, syncs, out = sample(lib, x, C, U, T, k, p, mp, *schedule)
        assert status == 0 and not (early and n), (schedule, status, n)
        check_row(x.float().numpy(), np.float32(U), full(T, 1.0), full(k, 0), np.float32(full(p, 1.0)),
                  np.float32(full(mp, 0.0)), *out)
        return syncs
    last = check(NOBODY, 0, 0)
    for lag, who in lags:
        for start in starts:
            if start <= last:
                check(lag, who, start)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("way", WAYS)
def test_ctas_that_fall_behind(emulated, way, dtype):
    """After any of the cluster's barriers, one CTA or all but one."""
    check_schedules(emulated, way, dtype, [(lag, who) for lag in (CTA, OTHERS) for who in range(C)],
                    range(1, 99), early=False)


@pytest.mark.parametrize("way", WAYS)
def test_a_warp_that_falls_behind(emulated, way):
    """The first and the last warp of the first CTA and of another."""
    check_schedules(emulated, way, torch.float32, [(WARP, w) for w in (0, 15, 21, 31)], (1, 2, 4, 8, 12),
                    early=False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("way", WAYS)
def test_ctas_that_start_late(emulated, way, dtype):
    """Nothing is stored into a CTA that has not begun or has ended: in BF16 the
    last CTA's part of the row is empty, so it is the first to store."""
    check_schedules(emulated, way, dtype, [(lag, who) for lag in (CTA, OTHERS) for who in range(C)], (0, 1, 2))
