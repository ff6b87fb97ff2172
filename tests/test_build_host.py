"""The build: one binding for each torch, and a library that does not wait for it."""

import os
import subprocess
import sys

import pytest
import torch

from vocab_ce_gb300 import build, step


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build in a folder of its own, of one translation unit."""
    monkeypatch.setattr(build, "LIB_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libtpce.so"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "SOURCES", ["ce_static.cu"])
    return tmp_path


def test_the_library_is_built_where_the_binding_cannot_be(elsewhere, monkeypatch):
    run = subprocess.run

    def without_gxx(cmd, *a, **k):
        if cmd[0] == "g++":
            return subprocess.CompletedProcess(cmd, 1, "", "no headers here")
        return run(cmd, *a, **k)

    monkeypatch.setattr(build.subprocess, "run", without_gxx)
    with pytest.raises(RuntimeError, match="no headers here"):
        build.build()
    assert os.path.exists(build.LIB_PATH)
    with pytest.raises(RuntimeError, match="no headers here"):    # and it is not taken for built the next time
        build.build()


def test_a_binding_of_another_torch_is_neither_loaded_nor_taken_for_built(elsewhere, monkeypatch):
    here = build.binding_path()
    assert torch.__version__ in here and os.path.dirname(here) == str(elsewhere)
    for path in (here, str(elsewhere / "_step_binding.so")):
        with open(path, "w") as f:
            f.write("of this torch")
    with open(build.LIB_PATH, "w") as f:
        f.write("")
    monkeypatch.setattr(torch, "__version__", "2.0.0+other")
    assert build.binding_path() != here
    monkeypatch.setattr(step, "_binding", None)
    with pytest.raises(RuntimeError, match="not built for this torch"):
        step._load()
    asked = []
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, *a, **k: asked.append(cmd[0]) or
                        subprocess.CompletedProcess(cmd, 1, "", "asked"))
    with pytest.raises(RuntimeError, match="asked"):
        build.build()
    assert asked == ["g++"]                                        # the library is current


def test_the_package_builds_without_importing_torch_first():
    # the module that builds the library is importable where torch is not
    code = "import sys; sys.modules['torch'] = None; import importlib.util as u; " \
           f"s = u.spec_from_file_location('b', {build.__file__!r}); m = u.module_from_spec(s); s.loader.exec_module(m)"
    assert subprocess.run([sys.executable, "-c", code], capture_output=True).returncode == 0
