"""The library is built where torch or its headers are missing (the C ABI needs neither); the tensor binding
is then left out, and says so when it is asked for.  CPU only; one small source stands for all of them."""
import importlib.util
import os
import types

import pytest

from paged_kv_cache_100_gb300 import build as B


@pytest.fixture
def small(monkeypatch, tmp_path):
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libpagedkv.so"))
    monkeypatch.setattr(B, "CU_SOURCES", [])
    return tmp_path


@pytest.mark.parametrize("torch", ["not installed", "without headers"])
def test_library_without_torch(small, monkeypatch, torch, capfd):
    real = importlib.util.find_spec
    fake = None if torch == "not installed" else types.SimpleNamespace(origin=str(small / "torch" / "__init__.py"))
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: fake if name == "torch" else real(name, *a))
    (small / B.BINDING_MODULE).write_text("of an earlier build")
    lib = B.build()
    assert os.path.exists(lib) and not os.path.exists(small / B.BINDING_MODULE)
    assert "not built" in capfd.readouterr().err
    made = os.path.getmtime(lib)
    assert B.build() == lib and os.path.getmtime(lib) == made          # not stale for want of the binding


def test_library_is_there_when_the_binding_does_not_compile(small, monkeypatch):
    bad = small / "bad.cpp"
    bad.write_text("this is not C++\n")
    monkeypatch.setattr(B, "BINDING", str(bad))
    with pytest.raises(RuntimeError, match="bad.cpp"):
        B.build()
    assert os.path.exists(B.LIB) and B._stale(B.LIB)                   # the next build tries again
