"""The native binding is loaded beside the torch that it was compiled against, and no
other."""
import pytest
import torch

from scaled_dot_product_06_gb300 import _native


@pytest.fixture
def fresh(monkeypatch):
    monkeypatch.setattr(_native, "_binding", None)


def test_of_this_torch(fresh):
    assert _native.binding().torch_version == torch.__version__
    assert _native.binding() is _native.binding()


def test_of_another_torch(fresh, monkeypatch):
    real = torch.__version__
    monkeypatch.setattr(torch, "__version__", "1.2.3")
    for _ in range(2):  # (nothing is kept of the first try)
        with pytest.raises(RuntimeError, match="compiled against torch " + real[:3] + ".*again beside torch 1.2.3"):
            _native.binding()


def test_that_does_not_load(fresh, monkeypatch, tmp_path):
    (tmp_path / "_binding.so").write_bytes(b"no shared object")
    monkeypatch.setattr(_native, "lib", lambda: None)
    monkeypatch.setattr(_native, "LIB_PATH", str(tmp_path / "libsdpa.so"))
    with pytest.raises(RuntimeError, match="does not load: build it again"):
        _native.binding()
    (tmp_path / "_binding.so").unlink()
    with pytest.raises(RuntimeError, match="is missing"):
        _native.binding()
