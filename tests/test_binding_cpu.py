"""The CPython extension is built against one torch and one Python: another one of either, or another
compiler command, builds it again, and it refuses to be used under another torch (no GPU needed)."""
import sys

import pytest

torch = pytest.importorskip("torch")
import ternary_quantized_moe_b200 as tq  # noqa: E402
from ternary_quantized_moe_b200 import build  # noqa: E402


@pytest.fixture
def built(tmp_path, monkeypatch):
    """An extension that is newer than its sources, with the key of this environment."""
    so, key = tmp_path / "_binding.so", tmp_path / "binding.key"
    so.write_bytes(b"")
    key.write_text(build._binding_key())
    monkeypatch.setattr(build, "BINDING", str(so))
    monkeypatch.setattr(build, "BINDING_KEY", str(key))
    return so, key


def test_current_extension_is_kept(built):
    assert not build._binding_stale()


def test_another_torch_builds_again(built, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert build._binding_stale()


def test_another_cxx11_abi_builds_again(built, monkeypatch):
    monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    assert build._binding_stale()


def test_another_python_builds_again(built, monkeypatch):
    class Other:
        cache_tag = "cpython-00"

    monkeypatch.setattr(sys, "implementation", Other)
    assert build._binding_stale()


def test_another_command_builds_again(built, monkeypatch):
    monkeypatch.setenv("CXX", "another-compiler")
    assert build._binding_stale()


def test_missing_key_or_extension_builds_again(built):
    so, key = built
    key.unlink()
    assert build._binding_stale()
    key.write_text(build._binding_key())
    so.unlink()
    assert build._binding_stale()


def test_extension_refuses_another_torch(monkeypatch):
    tq._bind()
    monkeypatch.setattr(tq, "_ext", None)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    with pytest.raises(ImportError, match="built with torch"):
        tq._bind()
