"""What a call on another stream than the current one allocates, with torch's CUDA
side replaced by a record of what it is asked (no GPU).
"""
from types import SimpleNamespace

import pytest
import torch

from scaled_dot_product_06_gb300 import api


class FakeStream:
    def __init__(self, name):
        self.name, self.cuda_stream, self.device = name, 7, torch.device("cpu")


@pytest.fixture
def cuda(monkeypatch):
    """[streams entered, (stream, bytes) allocations, (stream) notes of use]"""
    log = SimpleNamespace(current=[FakeStream("caller")], made=[], noted=[])

    class Entered:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            log.current.append(self.s)

        def __exit__(self, *_):
            log.current.pop()

    def empty(shape, dtype, device):
        log.made.append(log.current[-1].name)
        return SimpleNamespace(record_stream=lambda s: log.noted.append(s.name))

    monkeypatch.setattr(api.torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(api.torch.cuda, "current_stream", lambda device=None: log.current[-1])
    monkeypatch.setattr(api.torch.cuda, "stream", Entered)
    monkeypatch.setattr(api.torch, "empty", empty)
    return log


def test_memory_is_the_streams(cuda):
    dev = torch.device("cpu")
    api.new_tensor((4,), torch.float32, dev, None)
    assert cuda.made == ["caller"] and not cuda.noted
    side = FakeStream("side")
    api.new_tensor((4,), torch.float32, dev, side)
    assert cuda.made == ["caller", "side"] and cuda.noted == ["caller"]
    # a workspace is dropped at return: it goes back to its own stream at once
    api.new_tensor((4,), torch.uint8, dev, side, scratch=True)
    assert cuda.made[-1] == "side" and cuda.noted == ["caller"]
    # the current stream, named
    api.new_tensor((4,), torch.float32, dev, cuda.current[0])
    assert cuda.made[-1] == "caller" and cuda.noted == ["caller"]


def test_a_stream_of_another_device_is_refused():
    t = SimpleNamespace(device=torch.device("cuda", 0))
    assert api._stream_ptr(SimpleNamespace(cuda_stream=5, device=torch.device("cuda", 0)), t) == 5
    assert api._stream_ptr(SimpleNamespace(cuda_stream=5), t) == 5
    with pytest.raises(ValueError, match="device"):
        api._stream_ptr(SimpleNamespace(cuda_stream=5, device=torch.device("cuda", 1)), t)
