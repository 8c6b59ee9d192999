"""Host-side argument checks of the residual RMSNorm, rotary, slot-map and
sampling entry points, and the rotary frequencies (a host function); CPU only."""
import ctypes
import math

import pytest
import torch

import fp8_block_quantized_gb300 as jet
from fp8_block_quantized_gb300 import binding

OK, NULL, SHAPE, ALIGN, CUDA, DEVICE, WORKSPACE, TIMEOUT = range(8)
P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(16)]   # aligned, never dereferenced
MIS = ctypes.c_void_p(0x10008)
ODD = ctypes.c_void_p(0x10002)       # below any 4- or 8-byte type's alignment


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def swap(args, **kw):
    """args with the entries named _i replaced."""
    out = list(args)
    for k, v in kw.items():
        out[int(k[1:])] = v
    return out


def test_add_rmsnorm_quant(lib):
    f = lib.jet_add_rmsnorm_quant_1x128
    ok = [P[0], P[1], P[2], 4, 256, 1e-5, P[3], P[4], P[5], P[6], None]
    for i in (0, 1, 2, 6, 7, 8):
        assert f(*swap(ok, **{f"_{i}": None})) == NULL
        assert f(*swap(ok, **{f"_{i}": MIS})) == ALIGN
    assert f(*swap(ok, _9=ODD)) == ALIGN
    assert f(*swap(ok, _3=-1)) == SHAPE
    assert f(*swap(ok, _4=200)) == SHAPE
    assert f(*swap(ok, _4=1 << 24)) == SHAPE
    for eps in (-1.0, float("nan"), float("inf")):
        assert f(*swap(ok, _5=eps)) == SHAPE
    assert f(None, None, None, 0, 256, 1e-5, None, None, None, None, None) in (OK, DEVICE)


def test_add_rmsnorm_bwd(lib):
    f = lib.jet_add_rmsnorm_bwd
    need = lib.jet_workspace_bytes(binding.OP["add_rmsnorm_bwd"], 100, 0, 256)
    assert need == 100 * 256 * 4
    assert lib.jet_workspace_bytes(binding.OP["add_rmsnorm_bwd"], 10**6, 0, 4096) == 304 * 4096 * 4
    assert lib.jet_workspace_bytes(binding.OP["add_rmsnorm_bwd"], 10**6, 0, 256) == 1216 * 256 * 4
    assert lib.jet_workspace_bytes(binding.OP["add_rmsnorm_bwd"], 0, 0, 256) == 0
    ok = [P[0], P[1], P[2], P[3], P[4], P[5], P[6], 100, 256, P[7], P[8], P[9], need, None]
    for i in (0, 1, 2, 3, 9, 10):
        assert f(*swap(ok, **{f"_{i}": None})) == NULL
    for i in (0, 1, 3, 4, 5, 6, 9, 10, 11):
        assert f(*swap(ok, **{f"_{i}": MIS})) == ALIGN
    assert f(*swap(ok, _2=ODD)) == ALIGN
    assert f(*swap(ok, _7=-1)) == SHAPE
    assert f(*swap(ok, _8=100)) == SHAPE
    assert f(*swap(ok, _8=32768 + 128)) == SHAPE
    assert f(*swap(ok, _11=None)) == WORKSPACE
    assert f(*swap(ok, _12=need - 4)) == WORKSPACE


def test_rope(lib):
    f = lib.jet_rope
    ok = [P[0], 512, 4, P[1], 256, 2, 10, 128, 64, P[2], P[3], 0, 1.0, 0, P[4], 512, P[5], 256, None]
    for i in (0, 3, 9, 10, 14, 16):
        assert f(*swap(ok, **{f"_{i}": None})) == NULL
        assert f(*swap(ok, **{f"_{i}": ODD})) == ALIGN
    for i in (0, 3, 14, 16):
        assert f(*swap(ok, **{f"_{i}": MIS})) == ALIGN
    for i, v in ((1, 504), (4, 248), (15, 504), (17, 248), (2, -1), (2, 1025), (5, -1), (6, -1),
                 (6, 1 << 31), (7, 2048), (7, 100), (8, 130), (8, 63), (8, -2), (11, 2), (11, -1)):
        assert f(*swap(ok, **{f"_{i}": v})) == SHAPE, (i, v)
    for i in (1, 4, 15, 17):
        assert f(*swap(ok, **{f"_{i}": 516})) == ALIGN
    assert f(*swap(ok, _3=None, _5=0, _16=None)) in (OK, DEVICE) or torch.cuda.is_available()


def test_rope_kv_cache_write(lib):
    f = lib.jet_rope_kv_cache_write
    ok = [P[0], 512, 4, P[1], 256, P[2], 256, 2, 10, 128, 64, P[3], P[4], 0, 1.0, P[5], P[6], P[7],
          P[8], 512, P[9], P[10], 64, None]
    for i in (0, 3, 5, 11, 12, 15, 16, 17, 18, 20, 21):
        assert f(*swap(ok, **{f"_{i}": None})) == NULL, i
        assert f(*swap(ok, **{f"_{i}": ODD})) == ALIGN, i
    for i in (0, 3, 5, 18, 20, 21):
        assert f(*swap(ok, **{f"_{i}": MIS})) == ALIGN, i
    for i, v in ((1, 504), (4, 248), (6, 248), (19, 504), (8, -1), (9, 120), (10, 65), (13, 7),
                 (22, -1), (22, 1 << 41)):
        assert f(*swap(ok, **{f"_{i}": v})) == SHAPE, (i, v)


def test_kv_slot_map(lib):
    f = lib.jet_kv_slot_map
    ok = [P[0], P[1], 8, 16, P[2], 64, P[3], 100, P[4], 32, P[5], P[6], P[7], P[8], P[9], None]
    for i in (0, 1, 4, 6, 8, 10, 11, 12, 13, 14):
        assert f(*swap(ok, **{f"_{i}": None})) == NULL, i
        assert f(*swap(ok, **{f"_{i}": ODD})) == ALIGN, i
    for i, v in ((2, -1), (2, 8193), (3, 0), (3, 1 << 30), (5, -1), (5, 1 << 31), (7, -1), (9, -1)):
        assert f(*swap(ok, **{f"_{i}": v})) == SHAPE, (i, v)
    assert f(*swap(ok, _8=P[9])) == SHAPE                       # counts would overwrite free_next


def test_sample(lib):
    f = lib.jet_sample
    ok = [P[0], 0, 4, 1000, 1000, P[1], P[2], P[3], P[4], P[5], P[6], P[7], P[8], P[9], None]
    for i in (0, 5, 10, 11, 12, 13):
        assert f(*swap(ok, **{f"_{i}": None})) == NULL, i
    for i in (0, 5, 6, 7, 8, 9, 10, 11, 12, 13):
        assert f(*swap(ok, **{f"_{i}": ODD})) == ALIGN, i
    assert f(*swap(ok, _0=MIS)) == ALIGN
    for i, v in ((1, 2), (1, -1), (2, -1), (3, 0), (3, -5), (3, 262145), (4, 999)):
        assert f(*swap(ok, **{f"_{i}": v})) == SHAPE, (i, v)


def test_valid_arguments_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; this checks the no-device path")
    need = 100 * 256 * 4
    assert lib.jet_add_rmsnorm_quant_1x128(P[0], P[1], P[2], 4, 256, 1e-5, P[3], P[4], P[5], None,
                                           None) == DEVICE
    assert lib.jet_add_rmsnorm_bwd(P[0], P[1], P[2], P[3], None, None, None, 100, 256, P[7], P[8],
                                   P[9], need, None) == DEVICE
    assert lib.jet_rope(P[0], 512, 4, None, 0, 0, 10, 128, 64, P[2], P[3], 0, 1.0, 0, P[4], 512,
                        None, 0, None) == DEVICE
    assert lib.jet_rope_kv_cache_write(P[0], 512, 4, P[1], 256, P[2], 256, 2, 10, 128, 64, P[3],
                                       P[4], 0, 1.0, P[5], P[6], P[7], P[8], 512, P[9], P[10], 64,
                                       None) == DEVICE
    assert lib.jet_kv_slot_map(P[0], P[1], 8, 16, P[2], 64, P[3], 100, P[4], 32, P[5], P[6], P[7],
                               P[8], P[9], None) == DEVICE
    assert lib.jet_sample(P[0], 0, 4, 1000, 1000, P[1], None, None, None, None, P[6], P[7], P[8],
                          P[9], None) == DEVICE


def test_binding_refuses_wrong_tensors():
    """Type, shape and layout errors are raised before the library is called."""
    e = torch.empty
    x, g = e((4, 256), dtype=torch.bfloat16), e((256,), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        jet.add_rmsnorm_quant_1x128(x.float(), x, g)
    with pytest.raises(ValueError):
        jet.add_rmsnorm_quant_1x128(x, x[:2], g)
    with pytest.raises(ValueError):                                # a CPU tensor
        jet.add_rmsnorm_quant_1x128(x, x, g)
    with pytest.raises(ValueError):
        jet.add_rmsnorm_bwd(x, g, e((4,)), [])
    f, pos = e((32,), dtype=torch.float64), e((4,), dtype=torch.int64)
    q = e((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        jet.rope(q.float(), None, f, pos)
    with pytest.raises(ValueError):
        jet.rope(q, q[:3], f, pos)
    with pytest.raises(TypeError):
        jet.sample(e((4, 10), dtype=torch.float16), e((4,)))
    with pytest.raises(ValueError):
        jet.sample(e((10, 4)).t(), e((4,)))


# ---------------------------------------------------------------- frequencies

def ref_freq(R, base, scaling, factor, context, low, high):
    out = []
    for i in range(R // 2):
        f = base ** (-2 * i / R)
        if scaling == "linear":
            f /= factor
        elif scaling == "wavelength":
            turns = context * f / (2 * math.pi)
            if turns <= low:
                f = f / factor
            elif turns < high:
                s = (high - turns) / (high - low)
                f = f * (1 - s) + f * s / factor
        elif scaling == "ramp":
            at = lambda n: R * math.log(context / (2 * math.pi * n)) / (2 * math.log(base))
            a = min(max(math.floor(at(high)), 0), R - 1)
            b = min(max(math.ceil(at(low)), 0), R - 1)
            b = a + 0.001 if b <= a else b
            s = min(max((i - a) / (b - a), 0.0), 1.0)
            f = f * (1 - s) + f * s / factor
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


@pytest.mark.parametrize("R,base", [(2, 10000.0), (18, 10000.0), (128, 500000.0), (256, 1e6)])
@pytest.mark.parametrize("scaling", ["none", "linear", "wavelength", "ramp"])
def test_frequencies(R, base, scaling):
    got, mscale = jet.rope_inv_freq(R, base, scaling, 8.0, 8192.0, 1.0, 32.0, device="cpu")
    ref = ref_freq(R, base, scaling, 8.0, 8192.0, 1.0, 32.0)
    # pow within 1 ulp, a handful of binary64 operations after it
    assert ((got - ref).abs() <= 16 * 2.0 ** -53 * ref).all()
    want = 1 + 0.1 * math.log(8.0) if scaling == "ramp" else 1.0
    assert abs(mscale - want) <= 2.0 ** -24 * want
    if scaling == "wavelength" and R >= 128:
        plain = ref_freq(R, base, "none", 1, 1, 1, 2)
        assert got[0] == plain[0] and abs(got[-1] * 8 - plain[-1]) <= 1e-15   # ends: kept, divided


def test_frequency_refusals():
    for kw in (dict(R=7), dict(R=-2), dict(R=2048), dict(base=1.0), dict(base=float("nan")),
               dict(scaling="linear", factor=0.0), dict(scaling="wavelength", low=4.0, high=4.0),
               dict(scaling="ramp", low=-1.0), dict(scaling="ramp", context=0.0),
               dict(scaling="linear", factor=float("inf"))):
        args = dict(R=64, base=10000.0, scaling="none", factor=2.0, device="cpu") | kw
        with pytest.raises(jet.JetError) as e:
            jet.rope_inv_freq(**args)
        assert e.value.code == SHAPE, kw
