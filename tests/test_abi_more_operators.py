"""Host-side argument checks of the attention over the paged cache, the head's
log-probabilities and the gated activation's backward; CPU only."""
import ctypes

import pytest

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


def test_kv_attention(lib):
    f = lib.jet_kv_attention
    need = lib.jet_kv_attention_workspace(10, 8, 2, 128, 4, 2)
    assert need > 0
    #     q     ldq  T  Hq Hk  D    kc    vc   S    ks    vs   table width bs off lens B  po    pl   Ng
    ok = [P[0], 1024, 10, 8, 2, 128, P[1], P[2], 640, P[3], P[4], P[5], 7, 16, P[6], P[7], 4, P[8], P[9], 2,
          0.1, P[10], 1024, P[11], P[12], need, None]
    for i in (0, 6, 7, 9, 10, 11, 14, 15, 17, 18, 21):
        assert f(*swap(ok, **{f"_{i}": None})) == NULL, i
        assert f(*swap(ok, **{f"_{i}": ODD})) == ALIGN, i
    for i in (0, 6, 7, 21, 24):
        assert f(*swap(ok, **{f"_{i}": MIS})) == ALIGN, i
    assert f(*swap(ok, _23=ODD)) == ALIGN
    for i, v in ((1, 1016), (22, 1016), (2, -1), (2, 1 << 24), (3, 7), (3, 1026), (3, -8), (4, 0), (4, 3),
                 (5, 80), (5, 0), (5, 512), (8, -1), (8, 1 << 31), (12, -1), (12, 1 << 31), (13, 0),
                 (13, 1 << 30), (16, -1), (16, 8193), (19, -1), (19, 5), (20, 0.0), (20, -1.0),
                 (20, float("inf")), (20, float("nan"))):
        assert f(*swap(ok, **{f"_{i}": v})) == SHAPE, (i, v)
    for i in (1, 22):
        assert f(*swap(ok, **{f"_{i}": 1028})) == ALIGN
    assert f(*swap(ok, _24=None)) == WORKSPACE
    assert f(*swap(ok, _25=need - 1)) == WORKSPACE


def test_kv_attention_workspace(lib):
    f = lib.jet_kv_attention_workspace
    one = f(1, 8, 2, 128, 1, 0)
    assert one < f(1, 8, 2, 256, 1, 0)
    assert f(64, 8, 2, 128, 64, 4) >= one + 2 * 64 * 8 * 130 * 4
    for bad in ((-1, 8, 2, 128, 1, 0), (1, 8, 3, 128, 1, 0), (1, 8, 2, 96, 1, 0), (1, 8, 2, 128, 9000, 0),
                (1, 8, 2, 128, 1, 2), (0, 8, 2, 128, 1, 0), (1, 0, 0, 128, 1, 0), (1, 8, 2, 128, 0, 0)):
        assert f(*bad) == 0


def test_swiglu_bwd_quant(lib):
    f = lib.jet_swiglu_bwd_quant_1x128
    ok = [P[0], P[1], 512, P[2], 4, 256, P[3], P[4], P[5], P[6], None]
    for i in (0, 1, 3, 6, 7, 8, 9):
        assert f(*swap(ok, **{f"_{i}": None})) == NULL
        assert f(*swap(ok, **{f"_{i}": MIS})) == ALIGN
    for i, v in ((2, 248), (4, -1), (4, 1 << 31), (5, -128), (5, 200)):
        assert f(*swap(ok, **{f"_{i}": v})) == SHAPE
    assert f(*swap(ok, _2=516)) == ALIGN


def test_head_logp(lib):
    f = lib.jet_head_logp
    need = lib.jet_workspace_bytes(binding.OP["head_logp"], 100, 1000, 64)
    assert need > 0
    ok = [P[0], P[1], 100, 64, 1000, P[2], 1.0, P[3], P[4], P[5], need, None]
    for i in (0, 1, 5, 7, 8):
        assert f(*swap(ok, **{f"_{i}": None})) == NULL
        assert f(*swap(ok, **{f"_{i}": ODD})) == ALIGN
    for i in (0, 1, 9):
        assert f(*swap(ok, **{f"_{i}": MIS})) == ALIGN
    for i, v in ((2, -1), (2, 1 << 22), (3, 0), (3, 60), (3, 65544), (4, 0), (4, 1 << 24), (6, 0.0),
                 (6, -1.0), (6, float("inf")), (6, float("nan"))):
        assert f(*swap(ok, **{f"_{i}": v})) == SHAPE, (i, v)
    assert f(*swap(ok, _9=None)) == WORKSPACE
    assert f(*swap(ok, _10=need - 1)) == WORKSPACE


def test_head_logp_bwd(lib):
    f = lib.jet_head_logp_bwd
    need = lib.jet_workspace_bytes(binding.OP["head_logp_bwd"], 100, 1000, 64)
    assert need >= 100 * 1000 * 2
    ok = [P[0], P[1], 100, 64, 1000, P[2], P[3], P[4], 1.0, P[5], P[6], P[7], need, None]
    for i in (0, 1, 5, 6, 7):
        assert f(*swap(ok, **{f"_{i}": None})) == NULL
        assert f(*swap(ok, **{f"_{i}": ODD})) == ALIGN
    assert f(*swap(ok, _9=None, _10=None)) == NULL
    for i in (0, 1, 9, 10, 11):
        assert f(*swap(ok, **{f"_{i}": MIS})) == ALIGN
    for i, v in ((2, -1), (2, 1 << 22), (3, 0), (3, 60), (4, 0), (8, 0.0), (8, float("nan"))):
        assert f(*swap(ok, **{f"_{i}": v})) == SHAPE, (i, v)
    assert f(*swap(ok, _11=None)) == WORKSPACE
    assert f(*swap(ok, _12=need - 1)) == WORKSPACE


def test_head_workspaces(lib):
    f, op = lib.jet_workspace_bytes, binding.OP
    assert f(op["head_logp"], 0, 1000, 64) == 0 and f(op["head_logp"], 100, 1000, 60) == 0
    # d of a piece stays at half a gigabyte, or 4096 entries
    assert f(op["head_logp_bwd"], 4096, 128256, 512) < (1 << 30)
    assert f(op["head_logp_bwd"], 1 << 20, 128256, 64) < 2 * (4096 + 256) * (1 << 20) + 4 * (1 << 30)
