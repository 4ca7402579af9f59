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
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "_fp8b.so"))
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
    with open(elsewhere.BINDING_PATH, "w") as f:
        f.write("older")
    os.utime(elsewhere.BINDING_PATH, (1, 1))
    with pytest.warns(RuntimeWarning, match="_fp8b.so was not built"):
        assert elsewhere.build() == elsewhere.LIB_PATH
    assert os.path.exists(elsewhere.LIB_PATH) and not os.path.exists(elsewhere.BINDING_PATH)
    with pytest.raises(Exception):
        elsewhere.build_binding()


def test_module_is_built_beside_the_library(elsewhere):
    elsewhere.build()
    assert os.path.exists(elsewhere.BINDING_PATH)
    at = os.path.getmtime(elsewhere.BINDING_PATH)
    assert elsewhere.build() == elsewhere.LIB_PATH and elsewhere.build_binding() == elsewhere.BINDING_PATH
    assert os.path.getmtime(elsewhere.BINDING_PATH) == at      # (up to date: not built again)
