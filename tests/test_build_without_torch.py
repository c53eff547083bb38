"""The library needs nvcc only: where torch is not found it is made all the same, and the
tensor module is left out."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    from qwen3_gated_attention_gb300 import build
    build.build()


def _python(code, tmp_path):
    """Runs code in a process that finds no torch, with the outputs in tmp_path (objects of
    the last build are used again)."""
    head = f"""
import os, sys
class NoTorch:
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ModuleNotFoundError("No module named 'torch'", name="torch")
sys.meta_path.insert(0, NoTorch())
sys.path.insert(0, {ROOT!r})
from qwen3_gated_attention_gb300 import build, gattn
build.LIB = {str(tmp_path / "libgattn.so")!r}
build.MODULE = {str(tmp_path / "_paged.so")!r}
gattn.LIB_PATH = build.LIB
"""
    r = subprocess.run([sys.executable, "-c", head + code], capture_output=True, text=True, cwd=ROOT, timeout=900)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_the_library_is_built_and_loads(tmp_path):
    out = _python("assert build.build() == build.LIB\n"
                  "print(gattn.paged_attention_workspace(4, 2, 64, 1, 1))", tmp_path)
    assert int(out) > 0
    assert os.path.exists(tmp_path / "libgattn.so") and not os.path.exists(tmp_path / "_paged.so")


def test_the_entry_script_builds(tmp_path):
    _python("import __graft_entry__ as g\ng.build()", tmp_path)
    assert os.path.exists(tmp_path / "libgattn.so")


def test_the_library_comes_before_the_module(tmp_path, monkeypatch):
    """A module that does not compile is an error, with the library in place."""
    from qwen3_gated_attention_gb300 import build
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libgattn.so"))
    monkeypatch.setattr(build, "MODULE", str(tmp_path / "_paged.so"))
    monkeypatch.setattr(build, "_compile_module", lambda src: (str(tmp_path / "none.o"), "no such header"))
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()
    assert os.path.exists(build.LIB)


def test_calls_say_that_the_module_is_missing(monkeypatch):
    from qwen3_gated_attention_gb300 import device
    import qwen3_gated_attention_gb300 as package
    name = package.__name__ + "._paged"
    monkeypatch.delattr(package, "_paged", raising=False)
    monkeypatch.setitem(sys.modules, name, None)         # not found
    with pytest.raises(OSError, match="_paged.*is missing"):
        device._native("paged_rows")
