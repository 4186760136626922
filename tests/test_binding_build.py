"""The native half of the Python binding is tied to one torch and one interpreter: it is rebuilt when they change, and a
package that finds none for them loses the serving operators' calls alone."""
import importlib.util
import os
import subprocess
import sys
import types

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_rebuilt_for_another_torch_or_compiler(monkeypatch, tmp_path):
    spec = importlib.util.spec_from_file_location("hata_build_under_test", os.path.join(ROOT, "hash_aware_top_b200", "build.py"))
    B = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(B)
    built = []

    def run(cmd, **kw):
        built.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(B, "PKG", str(tmp_path))
    monkeypatch.setattr(B, "BINDING_LIB", str(tmp_path / "_serving.so.here"))
    monkeypatch.setattr(B, "BINDING_STAMP", str(tmp_path / "serving.json"), raising=False)
    monkeypatch.setattr(B, "subprocess", types.SimpleNamespace(run=run))
    B.build_binding()
    find, B.nvcc = B.nvcc, None  # what is up to date needs no compiler
    B.build_binding()
    assert len(built) == 1
    B.nvcc = find
    monkeypatch.setattr(torch, "__version__", "1.2.3+other")
    B.build_binding()
    B.build_binding()
    assert len(built) == 2 and any("1.2.3+other" in a for a in built[1])
    monkeypatch.setenv("CXX", "another-g++")
    B.build_binding()
    assert len(built) == 3 and built[2][0] == "another-g++"
    B.build_binding(force=True)
    os.remove(tmp_path / "_serving.so.here")
    B.build_binding()
    assert len(built) == 5


USE = """
import ctypes
import hash_aware_top_b200 as H
d = H.dims_for(1, 8, 2, 128, 128, 64, "bf16")
assert H.hata_workspace_size(d, 4) > 0 and H.hata_span_workspace_size(d, 1) > 0 and H.hata_version() > 0
f = ctypes.c_void_p(0x1000)
assert H.lib.hata_window_decode(ctypes.byref(d), None, f, f, f, 4, 0, 0.0, f, f, 1 << 40, None) == 1
try:
    H.hata_window_decode(d, None, None, None, None, 4, 0, 0.0, None, None)
except ImportError as e:
    assert "build.py" in str(e) and WHY in str(e), e
else:
    raise AssertionError("no ImportError")
"""


def run(before, why):
    r = subprocess.run([sys.executable, "-c", f"import sys, torch\nsys.path.insert(0, {ROOT!r})\nWHY = {why!r}\n{before}\n{USE}"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_a_native_half_that_cannot_be_loaded_loses_its_own_calls_alone():
    run("""
class Broken:
    def find_spec(self, name, path=None, target=None):
        if name == "hash_aware_top_b200._serving":
            raise ImportError("undefined symbol: of another torch")
sys.meta_path.insert(0, Broken())
""", "undefined symbol")


def test_a_native_half_of_another_torch_is_not_called():
    run("torch.__version__ = '0.0.1'", "0.0.1")


def test_the_native_half_here_is_for_this_torch():
    import hash_aware_top_b200 as H

    assert torch.__version__ in H._serving.built_for and sys.implementation.cache_tag in H._serving.built_for
    assert H._serving.__file__.endswith(".so") and sys.implementation.cache_tag.split("-")[1] in os.path.basename(H._serving.__file__)
