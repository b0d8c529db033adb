"""The build of the C library needs nvcc alone: what only the Python module needs may be missing."""
import os
import sysconfig

import pytest

from compressed_attention_cvq_b200 import build as B


@pytest.fixture(autouse=True)
def built():
    try:
        B.nvcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    B.build()
    if B._module_needs() is not None:
        pytest.skip("no module here to leave out")


@pytest.mark.parametrize("lack", ["compiler", "headers", "torch"])
def test_the_library_builds_without_what_the_module_needs(lack, monkeypatch, tmp_path, capsys):
    module = tmp_path / "_serving.so"
    module.write_bytes(b"of another build")
    monkeypatch.setattr(B, "MODULE", str(module))
    os.utime(module, (0, 0))                                     # older than its sources
    if lack == "compiler":
        monkeypatch.setenv("CXX", "a-compiler-that-is-not-there")
    elif lack == "headers":
        paths = dict(sysconfig.get_paths(), include=str(tmp_path))
        monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: paths)
    else:
        monkeypatch.setitem(__import__("sys").modules, "torch", None)
    assert B.build() == B.LIB
    assert not module.exists()                                   # importing it fails, and says why
    assert "not built" in capsys.readouterr().err


def test_a_module_of_these_sources_is_kept(monkeypatch):
    before = os.path.getmtime(B.MODULE)
    monkeypatch.setenv("CXX", "a-compiler-that-is-not-there")
    B.build()
    assert os.path.getmtime(B.MODULE) == before
