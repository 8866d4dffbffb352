"""What the binding must not pass on to a kernel: workspaces and keep bits that are not
the block of memory that their size says, on stand-ins for tensors (no GPU)."""
from types import SimpleNamespace

import pytest
import torch

from scaled_dot_product_06_gb300 import api


def test_workspace():
    cpu = torch.device("cpu")
    t = torch.empty(1024, dtype=torch.uint8)
    assert api.check_workspace(t, cpu) == (t.data_ptr(), 1024)
    f = torch.empty(16, 4)
    assert api.check_workspace(f, cpu) == (f.data_ptr(), 256)
    for bad in (t[::2], torch.empty(1, dtype=torch.uint8).expand(4096), f.t(), torch.empty(64, device="meta")):
        with pytest.raises(ValueError, match="workspace"):
            api.check_workspace(bad, cpu)


def words(n, **kw):
    return SimpleNamespace(**{"is_cuda": True, "dtype": torch.int32, "is_contiguous": lambda: True,
                              "numel": lambda: n, "data_ptr": lambda: 4096, **kw})


def test_keep_bits():
    need = api._words(0.25, 2, 4, 33, 64)
    assert need == 2 * 4 * 33 * 64 // 32 and api._words(0.25, 1, 1, 3, 20) == 2 and api._words(0.0, 2, 4, 33, 64) == 0
    w = api._window(True, None, False, None, 2, 4, words(need), words=need)
    assert w[-1] == 4096
    assert api._capped(20.0, True, None, False, None, None, 2, 4, words(need), need)[-1] == 4096
    for bad in (words(need - 1), words(need, is_cuda=False), words(need, dtype=torch.int64),
                words(need, is_contiguous=lambda: False)):
        with pytest.raises(ValueError, match="dropout_mask"):
            api._window(True, None, False, None, 2, 4, bad, words=need)
        with pytest.raises(ValueError, match="dropout_mask"):
            api._capped(20.0, True, None, False, None, None, 2, 4, bad, need)


def test_check_io():
    def t(**kw):
        return SimpleNamespace(**{"is_cuda": True, "shape": torch.Size((2, 3)), "dtype": torch.float16,
                                  "is_contiguous": lambda: True, **kw})
    api._check_io("x", t(), (2, 3), torch.float16)
    for bad, what in ((t(is_cuda=False), "CUDA"), (t(shape=torch.Size((3, 2))), "shape"),
                      (t(dtype=torch.bfloat16), "dtype"), (t(is_contiguous=lambda: False), "contiguous")):
        with pytest.raises(ValueError, match=what):
            api._check_io("x", bad, (2, 3), torch.float16)
