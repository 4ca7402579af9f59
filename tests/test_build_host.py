"""Host-side checks of the build: what the C library needs, and what only the
compiled Python module does."""
import os
import sys

import pytest

pytest.importorskip("torch")


@pytest.fixture()
def elsewhere(monkeypatch, tmp_path):
    """The build module with the library up to date and its Python module's path
    and objects in a folder of the test's."""
    from expert_routed_ffn_selectedsoftmax_gb300 import build
    build.build()
    monkeypatch.setattr(build, "binding_path", lambda: str(tmp_path / "_fp8b.so"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    return build


@pytest.mark.parametrize("missing", ["compiler", "torch"])
def test_library_builds_where_the_module_cannot(elsewhere, monkeypatch, missing):
    """Without a host compiler or without PyTorch build() still gives the library,
    with a warning; a module of older sources does not stay; build_binding raises."""
    if missing == "compiler":
        monkeypatch.setenv("CXX", "/nonexistent/c++")
    else:
        monkeypatch.setitem(sys.modules, "torch", None)
    with open(elsewhere.binding_path(), "w") as f:
        f.write("older")
    os.utime(elsewhere.binding_path(), (1, 1))
    with pytest.warns(RuntimeWarning, match="_fp8b. was not built"):
        assert elsewhere.build() == elsewhere.LIB_PATH
    assert os.path.exists(elsewhere.LIB_PATH) and not os.path.exists(elsewhere.binding_path())
    with pytest.raises(Exception):
        elsewhere.build_binding()


def test_module_is_built_beside_the_library(elsewhere):
    elsewhere.build()
    assert os.path.exists(elsewhere.binding_path())
    at = os.path.getmtime(elsewhere.binding_path())
    assert elsewhere.build() == elsewhere.LIB_PATH and elsewhere.build_binding() == elsewhere.binding_path()
    assert os.path.getmtime(elsewhere.binding_path()) == at      # (up to date: not built again)


def test_module_belongs_to_one_pytorch_and_python(monkeypatch):
    """An interpreter or a PyTorch of another version does not find this one's
    module: it counts as not built, and the calls say what to do."""
    import sysconfig

    import torch

    from expert_routed_ffn_selectedsoftmax_gb300 import binding, build
    build.build()
    mine = build.binding_path()
    assert os.path.exists(mine) and build.binding_up_to_date()
    assert torch.__version__ in mine and mine.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(binding, "_fp8b_module", None)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1+other")
        assert build.binding_path() != mine and not build.binding_up_to_date()
        with pytest.raises(RuntimeError, match="build it for this PyTorch"):
            binding.moe_quant_fp8b(torch.zeros(1, 16))
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: ".cpython-30-other.so")
        assert build.binding_path() != mine and not build.binding_up_to_date()
    with pytest.raises(ValueError, match="CUDA"):      # (the right one is loaded again)
        binding.moe_quant_fp8b(torch.zeros(1, 16))
