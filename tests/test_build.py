"""The library and the binding's extension module are built and loaded apart; CPU only."""
import pytest
import torch

import fp8_block_quantized_gb300 as jet
from fp8_block_quantized_gb300 import binding, build


@pytest.fixture
def no_module(monkeypatch, tmp_path):
    """Nothing loaded, and an extension module that is not there and cannot be built."""
    def fail(*args, **kw):
        raise RuntimeError("no headers to build it with")
    binding.load()
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "_marshal", None)
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(build, "build_marshal", fail)


def test_the_library_loads_without_the_module(no_module):
    assert binding.load().jet_version() > 0
    assert jet.binding.workspace_bytes("add_rmsnorm_bwd", 4, 0, 256) == 4 * 256 * 4


def test_the_operators_say_what_is_missing(no_module):
    q, f, pos = torch.empty((0, 2, 64), dtype=torch.bfloat16), torch.empty((32,), dtype=torch.float64), \
        torch.empty((0,), dtype=torch.int64)
    for _ in range(2):                 # and again: the first failure leaves nothing half loaded
        with pytest.raises(RuntimeError, match="no headers"):
            jet.jet_rope(q, None, f, pos, q, None)
    assert binding.load().jet_version() > 0


def test_the_library_is_built_without_the_module(no_module):
    with pytest.warns(UserWarning, match="no headers"):
        assert build.build() == build.LIB


def test_another_torch_or_python_has_a_module_of_its_own(monkeypatch):
    """The module holds one torch's and one interpreter's binary interface: after a
    change of either the one built before is not taken for current."""
    import importlib.metadata
    import importlib.util
    import sysconfig

    def path_under(torch_version, suffix):
        with monkeypatch.context() as m:
            version, var = importlib.metadata.version, sysconfig.get_config_var
            m.setattr(importlib.metadata, "version", lambda n: torch_version if n == "torch" else version(n))
            m.setattr(sysconfig, "get_config_var", lambda n: suffix if n == "EXT_SUFFIX" else var(n))
            spec = importlib.util.spec_from_file_location("build_again", build.__file__)
            again = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(again)
            return again.MARSHAL
    here = sysconfig.get_config_var("EXT_SUFFIX")
    assert path_under(importlib.metadata.version("torch"), here) == build.MARSHAL
    paths = {build.MARSHAL, path_under("1.0+cu0", here), path_under("1.0+cu0", ".cpython-39-x.so")}
    assert len(paths) == 3
