"""What the build needs: nvcc for the library, torch and a host compiler for the Python module
alone (stand-ins for the compilers, no GPU)."""
import importlib.util
import os

import pytest

from paged_kv_attention_18_gb300 import build as B

TOUCH = """#!/bin/sh
while [ $# -gt 0 ]; do [ "$1" = -o ] && echo made > "$2"; shift; done
"""


@pytest.fixture
def place(tmp_path, monkeypatch):
    def script(name, text):
        path = tmp_path / name
        path.write_text(text)
        path.chmod(0o755)
        return str(path)

    monkeypatch.setattr(B, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libpagedserve.so"))
    monkeypatch.setattr(B, "NATIVE", str(tmp_path / "_native.so"))
    monkeypatch.setenv("NVCC", script("nvcc", TOUCH))
    monkeypatch.setenv("CXX", script("cxx", TOUCH))
    return script


def test_both(place):
    assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and os.path.exists(B.NATIVE)


def test_without_torch_the_library_alone(place, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setenv("CXX", "/no/such/compiler")
    assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.NATIVE)


@pytest.mark.parametrize("missing", [False, True])
def test_without_a_host_compiler_the_library_is_there(place, monkeypatch, missing):
    monkeypatch.setenv("CXX", "/no/such/compiler" if missing else place("bad", "#!/bin/sh\nexit 1\n"))
    with pytest.raises((RuntimeError, OSError)):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.NATIVE)
