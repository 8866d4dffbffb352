"""What build() makes and in which order, with the compilers replaced by stand-ins: the
library does not need torch, and does not wait for its binding."""
import importlib.util
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(monkeypatch, tmp_path):
    """build.py on its own, as a host without torch runs it; steps: what was made."""
    spec = importlib.util.spec_from_file_location(
        "build_alone", os.path.join(ROOT, "scaled_dot_product_06_gb300", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    b.steps, b.broken = [], set()

    def run(cmd, what):
        if what in b.broken:
            raise RuntimeError(what + " failed")
        b.steps.append(what)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(what)

    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "_compile", lambda src, verbose: src)
    monkeypatch.setattr(b, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    for name, at in (("BUILD", "_build"), ("LIB", "libsdpa.so"), ("BINDING", "_binding.so")):
        monkeypatch.setattr(b, name, str(tmp_path / at))
    return b


def test_without_torch(build, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    with open(build.BINDING, "w") as f:
        f.write("of another build")
    assert build.build() == build.LIB
    assert build.steps == ["link of libsdpa.so"] and os.path.exists(build.LIB)
    assert not os.path.exists(build.BINDING)
    assert "_binding.so is left out" in capsys.readouterr().err


def test_a_binding_that_fails_leaves_the_library(build):
    for what in ("g++ on binding.cpp", "link of _binding.so"):
        build.broken = {what}
        build.steps.clear()
        if os.path.exists(build.LIB):
            os.remove(build.LIB)
        with pytest.raises(RuntimeError, match="failed"):
            build.build()
        assert "link of libsdpa.so" in build.steps and os.path.exists(build.LIB)
        assert not os.path.exists(build.BINDING)


def test_with_torch(build):
    build.build()
    assert sorted(build.steps[:2]) == ["g++ on binding.cpp", "link of libsdpa.so"]
    assert build.steps[2:] == ["link of _binding.so"]
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING)
