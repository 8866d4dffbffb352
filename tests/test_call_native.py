"""Calls through the native binding, with it and torch's CUDA side replaced by
stand-ins (no GPU): the stream they run on, what is noted of their outputs, statuses,
and that no binding launches in another way."""
import ast
import inspect
import os
import re
from types import SimpleNamespace

import pytest
import torch

from scaled_dot_product_06_gb300 import _native, api, paged, prefix, rows

CSRC = os.path.join(os.path.dirname(os.path.abspath(_native.__file__)), "csrc")


class FakeStream:
    def __init__(self, name, device=0):
        self.name, self.cuda_stream, self.device = name, 7, torch.device("cuda", device)


@pytest.fixture
def native(monkeypatch):
    """ran: (stream, arguments) of calls; noted: (output, stream); out: what a call returns."""
    log = SimpleNamespace(current=[FakeStream("caller")], ran=[], noted=[], out=None, checked=[])

    class Entered:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            log.current.append(self.s)

        def __exit__(self, *_):
            log.current.pop()

    def entry(*args):
        log.ran.append((log.current[-1].name, args))
        if isinstance(log.out, Exception):
            raise log.out
        return log.out

    log.tensor = lambda name: SimpleNamespace(record_stream=lambda s: log.noted.append((name, s.name)))
    log.on = SimpleNamespace(is_cuda=True, device=torch.device("cuda", 0))
    monkeypatch.setattr(api._native, "binding", lambda: SimpleNamespace(entry=entry))
    monkeypatch.setattr(api._native, "check", lambda st, what: log.checked.append((st, what)))
    monkeypatch.setattr(api.torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(api.torch.cuda, "ExternalStream", lambda ptr, device: FakeStream(f"external {ptr}"))
    monkeypatch.setattr(api.torch.cuda, "current_stream", lambda device=None: log.current[-1])
    monkeypatch.setattr(api.torch.cuda, "stream", Entered)
    return log


def test_the_current_stream(native):
    native.out = (native.tensor("a"), None)
    assert api.call_native("entry", None, native.on, (None, None), 1, 2) is native.out
    assert native.ran == [("caller", (1, 2))] and not native.noted and not native.checked


def test_another_stream(native):
    native.out = tuple(native.tensor(n) for n in "abc") + (None,)
    given = (None, native.out[1], None, None)
    assert api.call_native("entry", FakeStream("side"), native.on, given, 3) is native.out
    # allocated and run there; what the call made is the caller's too, what was given is not noted
    assert native.ran == [("side", (3,))] and native.noted == [("a", "caller"), ("c", "caller")]
    assert [s.name for s in native.current] == ["caller"]
    # a handle, and the current stream by its name
    api.call_native("entry", SimpleNamespace(cuda_stream=9), native.on, given)
    assert native.ran[-1][0] == "external 9" and len(native.noted) == 4
    api.call_native("entry", native.current[0], native.on, given)
    assert native.ran[-1][0] == "caller" and len(native.noted) == 4


def test_streams_that_do_not_fit(native):
    with pytest.raises(ValueError, match="device"):
        api.call_native("entry", FakeStream("far", 1), native.on, ())
    with pytest.raises(ValueError, match="not on a CUDA device"):
        api.call_native("entry", FakeStream("side"), SimpleNamespace(is_cuda=False, device=torch.device("cpu")), ())
    assert not native.ran


def test_statuses_and_errors(native):
    native.out = 4
    for stream in (None, FakeStream("side")):
        api.call_native("entry", stream, native.on, (None,))
    assert native.checked == [(4, "sdpa_entry")] * 2 and not native.noted
    native.out = ValueError("refused")
    with pytest.raises(ValueError, match="refused"):
        api.call_native("entry", FakeStream("side"), native.on, (None,))
    assert [s.name for s in native.current] == ["caller"]


def test_every_launch_goes_that_way():
    """The Python bindings launch through _run or call_native, and the native one calls the
    entry points on the stream of the guarded device only."""
    binders = []
    for module in (api, paged, prefix, rows):
        tree = ast.parse(inspect.getsource(module))
        for node in ast.walk(tree):
            if isinstance(node, ast.Attribute) and isinstance(node.value, ast.Call) \
                    and ast.unparse(node.value.func) == "_native.lib":
                assert "workspace_size" in node.attr or node.attr in ("sdpa_device_error", "sdpa_debug_fault"), node.attr
        binders += [f.name for f in ast.walk(tree) if isinstance(f, ast.FunctionDef) and "_native.binding" in ast.unparse(f)]
    assert binders == ["call_native"]
    with open(os.path.join(CSRC, "binding.cpp")) as f:
        source = re.sub(r"//[^\n]*", "", f.read())
    calls = re.findall(r"\b(sdpa_\w+)\(([^;]*)\);", source)
    launches = [c for c in calls if not c[0].endswith("_workspace_size")]
    assert {c[0] for c in launches} == {"sdpa_page_slots", "sdpa_fwd_paged", "sdpa_qk_norm_rope", "sdpa_qk_norm_rope_paged"}
    assert all(re.search(r",\s*stream$", args) for _, args in launches)
    # the one stream that is not a parameter: the current one of the device made current just before
    bodies = source.split("sdpa_status_t call(")
    assert len(bodies) == 2 and source.count("void* stream =") == 1
    own = bodies[1]
    assert own.index("CUDAGuard device(") < own.index("void* stream = c10::cuda::getCurrentCUDAStream(") < own.index("entry(stream)")
    assert source.count("= call(at, [&](void* stream)") == 3
