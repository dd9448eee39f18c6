"""What build() makes of which machine.  A one-line library stands in for the
real one, in a folder of its own."""
import os
from types import SimpleNamespace

import pytest

from zero_optimizer_step_rs_gb300 import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    source = tmp_path / "one.cpp"
    source.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "SOURCES", [str(source)])
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libone.so"))
    monkeypatch.setattr(build, "EXT", str(tmp_path / "_lm.so"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "build"))
    return tmp_path


def installed(monkeypatch, folder):
    """As if torch were installed in that folder (None: nowhere)."""
    spec = folder and SimpleNamespace(submodule_search_locations=[str(folder)])
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: spec)


def test_the_library_is_built_without_torch(small, monkeypatch, capsys):
    installed(monkeypatch, None)
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.EXT)
    assert "no torch" in capsys.readouterr().err
    before = os.path.getmtime(build.LIB)
    build.build()                                        # nothing left to do
    assert os.path.getmtime(build.LIB) == before


def test_the_library_is_built_beside_a_torch_without_cuda(small, monkeypatch):
    (small / "torch" / "lib").mkdir(parents=True)
    installed(monkeypatch, small / "torch")
    build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.EXT)


def test_a_module_that_does_not_compile_leaves_the_library(small, monkeypatch):
    bad = small / "bad.cpp"
    bad.write_text("#error no\n")
    monkeypatch.setattr(build, "EXT_SOURCE", str(bad))
    with pytest.raises(RuntimeError, match="#error no"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.EXT)


def test_the_module_is_built_again_for_another_torch(monkeypatch, tmp_path):
    """The one that stands here, as build() leaves it, is fresh for the installed
    torch and stale for another version of it, or the same one elsewhere."""
    build.build()
    if build.torch_dir() is None:
        pytest.skip("no torch with CUDA here")
    assert not build._stale()
    (tmp_path / "lib").mkdir()
    (tmp_path / "lib" / "libc10_cuda.so").write_text("")
    (tmp_path / "version.py").write_text("__version__ = '0.0'\n")
    installed(monkeypatch, tmp_path)
    assert build._stale()
