"""The build step: the C-ABI library needs nvcc alone, whatever becomes of the Python binding."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# build.py as a script would run it, with its outputs in a folder of their own and one unit of the library
CHILD = """
import importlib.util, os, sys
spec = importlib.util.spec_from_file_location("build", sys.argv[1])
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
out = sys.argv[2]
b.BUILD, b.LIB, b.BIND, b.SOURCES = out, os.path.join(out, "lib.so"), os.path.join(out, "bind.so"), ["planner.cpp"]
b.BIND_FOR = os.path.join(out, "bind.for")
"""


def child(tmp_path, code):
    script = os.path.join(ROOT, "mixed_lora_projection_gb300", "build.py")
    return subprocess.run([sys.executable, "-c", CHILD + code, script, str(tmp_path)], capture_output=True, text=True)


def test_library_builds_without_pytorch(tmp_path):
    r = child(tmp_path, "sys.modules['torch'] = None\nb.build()\nassert not b._stale()\n")
    assert r.returncode == 0, r.stderr
    assert (tmp_path / "lib.so").exists() and not (tmp_path / "bind.so").exists()


def test_library_is_linked_whatever_becomes_of_the_binding(tmp_path):
    (tmp_path / "broken.cpp").write_text("#error not this one\n")
    r = child(tmp_path, "b.BIND_SOURCE = os.path.join(out, 'broken.cpp')\nb.build()\n")
    assert r.returncode != 0 and "not this one" in r.stderr
    assert (tmp_path / "lib.so").exists() and not (tmp_path / "bind.so").exists()


def test_binding_of_another_pytorch_is_stale_and_refused(lib, tmp_path, monkeypatch):
    from mixed_lora_projection_gb300 import build, layer
    assert not build._stale()
    layer._load()
    monkeypatch.setattr(layer, "_bind", None)
    monkeypatch.setattr(layer, "bind_for", lambda: "PyTorch 1.0, cpython-30")
    with pytest.raises(RuntimeError, match="not built for this PyTorch"):
        layer._load()
    assert layer._bind is None
    other = tmp_path / "for"
    monkeypatch.setattr(build, "BIND_FOR", str(other))
    assert build._stale()                                      # one that does not say
    other.write_text("PyTorch 1.0, cpython-30")
    assert build._stale()
