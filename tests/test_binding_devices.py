"""Calls on tensors of another device than the current one, with torch's CUDA side and
the library replaced by stand-ins (no GPU): the tensors' device is current during
the call, and operands of two devices are refused."""
import ast
import inspect
from types import SimpleNamespace

import pytest
import torch

from scaled_dot_product_06_gb300 import api, prefix, rows


def test_device_is_current_during_the_call(monkeypatch):
    now = [0]
    seen = []

    class Device:
        def __init__(self, d):
            self.d = d.index

        def __enter__(self):
            now.append(self.d)

        def __exit__(self, *_):
            now.pop()

    lib = SimpleNamespace(sdpa_fwd_gqa=lambda *a: seen.append((now[-1], a)) or 0, bad=lambda *a: 1)
    monkeypatch.setattr(api._native, "lib", lambda: lib)
    monkeypatch.setattr(api.torch.cuda, "current_device", lambda: now[-1])
    monkeypatch.setattr(api.torch.cuda, "device", Device)
    for d in (0, 1):
        t = SimpleNamespace(device=torch.device("cuda", d), get_device=lambda d=d: d)
        api._run(t, "sdpa_fwd_gqa", 5, 6)
        assert seen[-1] == (d, (5, 6)) and now == [0]
        monkeypatch.setattr(api._native, "check", lambda st, what: seen.append((st, what)))
        api._run(t, "bad")
        assert seen[-1] == (1, "bad")


def test_operands_of_two_devices():
    one, two = torch.device("cuda", 0), torch.device("cuda", 1)

    def t(device):
        return SimpleNamespace(is_cuda=True, device=device, shape=torch.Size((2, 3)), dtype=torch.float16,
                               is_contiguous=lambda: True)
    api._check_io("k", t(one), (2, 3), torch.float16, one)
    with pytest.raises(ValueError, match="device of q"):
        api._check_io("k", t(two), (2, 3), torch.float16, one)
    api._check_device(one, mask=None, seqstart_q=t(one))
    with pytest.raises(ValueError, match="seqstart_q must be on the device of q"):
        api._check_device(one, mask=None, seqstart_q=t(two))


def test_every_launch_goes_that_way():
    """No binding calls a launching entry point past _run."""
    for module in (api, prefix, rows):
        for node in ast.walk(ast.parse(inspect.getsource(module))):
            if isinstance(node, ast.Attribute) and isinstance(node.value, ast.Call) \
                    and ast.unparse(node.value.func) == "_native.lib":
                assert "workspace_size" in node.attr or node.attr in ("sdpa_device_error", "sdpa_debug_fault"), node.attr
