"""Refusals of the shared-prefix attention on the CPU, before any CUDA call,
and the sizes of its workspace."""
import ctypes

import pytest
import torch

from scaled_dot_product_06_gb300 import _native, sdpa_fwd_prefix
from test_abi import MIS, NULL, P, lib  # noqa: F401

BAD, UNS, ALIGN, WS, OK = (_native.SDPA_ERR_INVALID_ARG, _native.SDPA_ERR_UNSUPPORTED,
                           _native.SDPA_ERR_MISALIGNED, _native.SDPA_ERR_WORKSPACE, _native.SDPA_OK)


def fwd(lib, b=2, h=4, h_kv=2, s_q=1, s_p=100, s_max=50, d=64, d_v=64, scale=0.125, cap=0.0, dtype=0, q=P,
        kp=P, vp=P, k=P, v=P, lens=P, o=P, lse=P, ws=P, nbytes=1 << 40):
    return lib.sdpa_fwd_prefix(b, h, h_kv, s_q, s_p, s_max, d, d_v, scale, cap, dtype, q, kp, vp, k, v, lens, o,
                               lse, ws, nbytes, None)


def test_refusals(lib):  # noqa: F811
    for kw in (dict(b=-1), dict(s_max=-1), dict(s_p=-5), dict(h_kv=3), dict(h_kv=0), dict(scale=float("nan")),
               dict(cap=-1.0), dict(cap=5000.0), dict(cap=float("nan")), dict(q=NULL), dict(o=NULL),
               dict(lse=NULL), dict(kp=NULL), dict(vp=NULL), dict(k=NULL), dict(v=NULL), dict(lens=NULL)):
        assert fwd(lib, **kw) == BAD, kw
    for kw in (dict(dtype=3), dict(d=96), dict(d=192, d_v=192), dict(s_max=1 << 40), dict(s_p=1 << 30),
               dict(b=1 << 20, s_q=1 << 20)):
        assert fwd(lib, **kw) == UNS, kw
    for kw in (dict(q=MIS), dict(kp=MIS), dict(v=MIS), dict(o=MIS), dict(ws=MIS),
               dict(lens=ctypes.c_void_p((1 << 20) + 1))):
        assert fwd(lib, **kw) == ALIGN, kw
    assert fwd(lib, ws=NULL) == WS
    assert fwd(lib, nbytes=100) == WS
    for kw in (dict(b=0), dict(s_q=0), dict(h=0, h_kv=0)):
        assert fwd(lib, q=NULL, o=NULL, **kw) == OK, kw


def test_workspace_size(lib):  # noqa: F811
    size = lib.sdpa_fwd_prefix_workspace_size
    assert size(2, 4, 2, 1, 0, 0, 64, 64) == 0  # no key at all
    # one key tile each: two slots of the prefix and eight of the own keys, 8 rows
    assert size(2, 4, 2, 1, 100, 50, 64, 64) == (10 * 8 * 65 * 4 + 255) // 256 * 256
    assert size(2, 4, 3, 1, 100, 50, 64, 64) == 0
    assert size(2, 4, 2, 1, 100, 50, 96, 96) == 0


def test_binding_refusals():
    q = torch.zeros(1, 2, 1, 64).half()
    p, c = torch.zeros(1, 8, 64).half(), torch.zeros(1, 1, 8, 64).half()
    n = torch.zeros(1, dtype=torch.int32)
    for a in ((q, p, p, c, c, n), (q[0], p, p, c, c, n), (q, c, p, c, c, n), (q.float(), p, p, c, c, n)):
        with pytest.raises(ValueError):
            sdpa_fwd_prefix(*a)
