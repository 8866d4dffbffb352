"""Refusals of the attention over a paged cache on the CPU, before any CUDA call,
and the size of its workspace."""
import ctypes

import pytest
import torch

from scaled_dot_product_06_gb300 import _native, sdpa_fwd_paged, sdpa_fwd_paged_workspace_size
from test_abi import MIS, NULL, P, lib  # noqa: F401

BAD, UNS, ALIGN, WS, OK = (_native.SDPA_ERR_INVALID_ARG, _native.SDPA_ERR_UNSUPPORTED,
                           _native.SDPA_ERR_MISALIGNED, _native.SDPA_ERR_WORKSPACE, _native.SDPA_OK)


def rows_of(ptr=1 << 20, st=(2048, 64, 1024)):
    return ctypes.byref(_native.Rows(ptr, *st))


def fwd(lib, b=2, h=4, h_kv=2, s_q=1, d=64, d_v=64, scale=0.125, cap=0.0, left=-1, dtype=0, q=P, k=None, v=None,
        n_pages=50, page=16, table=P, wide=70, stride=70, lens=P, o=P, lse=P, ws=P, nbytes=1 << 40):
    return lib.sdpa_fwd_paged(b, h, h_kv, s_q, d, d_v, scale, cap, left, dtype, q, k or rows_of(), v or rows_of(),
                              n_pages, page, table, wide, stride, lens, o, lse, ws, nbytes, None)


def test_refusals(lib):  # noqa: F811
    for kw in (dict(b=-1), dict(s_q=-1), dict(h_kv=3), dict(h_kv=0), dict(n_pages=-1), dict(wide=-1),
               dict(stride=69), dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0), dict(cap=5000.0),
               dict(cap=float("nan")), dict(scale=1e38, cap=1e-3), dict(q=NULL), dict(o=NULL), dict(lse=NULL),
               dict(table=NULL), dict(lens=NULL), dict(k=rows_of(ptr=None)), dict(v=rows_of(ptr=None)),
               dict(k=rows_of(st=(0, 64, 1024))), dict(v=rows_of(st=(2048, -64, 1024))),
               dict(v=rows_of(st=(2048, 64, 1 << 40)))):
        assert fwd(lib, **kw) == BAD, kw
    for kw in (dict(dtype=3), dict(d=96), dict(d=192, d_v=192), dict(page=12), dict(page=4), dict(page=0),
               dict(page=1 << 21), dict(n_pages=1 << 30), dict(wide=1 << 26, stride=1 << 26),
               dict(b=1 << 20, s_q=1 << 20), dict(stride=1 << 50),
               dict(b=1 << 20, h=8, h_kv=8, wide=1 << 14, stride=1 << 14)):
        assert fwd(lib, **kw) == UNS, kw
    for kw in (dict(q=MIS), dict(o=MIS), dict(lse=MIS), dict(ws=MIS), dict(k=rows_of(ptr=(1 << 20) + 8)),
               dict(v=rows_of(st=(2048, 60, 1024))), dict(k=rows_of(st=(2052, 64, 1024))),
               dict(lens=ctypes.c_void_p((1 << 20) + 1)), dict(table=ctypes.c_void_p((1 << 20) + 2))):
        assert fwd(lib, **kw) == ALIGN, kw
    assert fwd(lib, ws=NULL) == WS
    assert fwd(lib, nbytes=100) == WS
    assert fwd(lib, wide=32, stride=32, ws=NULL, nbytes=0, q=NULL) == BAD  # (it needs none)
    for kw in (dict(b=0), dict(s_q=0), dict(h=0, h_kv=1)):
        assert fwd(lib, q=NULL, o=NULL, **kw) == OK, kw


def test_workspace_size(lib):  # noqa: F811
    size = lib.sdpa_fwd_paged_workspace_size
    for h, h_kv, s_q, rows in ((8, 8, 1, 8), (16, 1, 1, 16), (32, 2, 1, 16), (32, 2, 2, 32), (33, 1, 1, 64), (64, 1, 8, 64)):
        # two slots a CTA, rows of d_v + 1 floats, and six words a CTA
        assert size(h, h_kv, s_q, 64, 64, 16, 33) == (304 * rows * 65 * 4 + 6 * 152 * 8 + 255) // 256 * 256
        assert sdpa_fwd_paged_workspace_size(h, h_kv, s_q, 192, 128, 1024, 7) == (304 * rows * 129 * 4 + 6 * 152 * 8 + 255) // 256 * 256
        # up to four key tiles a sequence: nothing to join
        assert size(h, h_kv, s_q, 64, 64, 16, 32) == 0 and size(h, h_kv, s_q, 64, 64, 128, 0) == 0
    for bad in ((8, 3, 1, 64, 64, 16, 99), (8, 2, 1, 96, 96, 16, 99), (8, 2, 0, 64, 64, 16, 99), (8, 2, 1, 64, 64, 0, 99),
                (8, 2, 1, 64, 64, 16, -1), (8, 2, 1, 64, 64, 1 << 40, 1 << 40)):
        assert size(*bad) == 0, bad


def test_binding_refusals():
    q, pages = torch.zeros(1, 2, 1, 64).half(), torch.zeros(4, 1, 16, 64).half()
    n, t = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 3, dtype=torch.int32)
    for a in ((q, pages, pages, t, n), (q[0], pages, pages, t, n), (q, pages[0], pages, t, n),
              (q.float(), pages, pages, t, n)):
        with pytest.raises(ValueError):
            sdpa_fwd_paged(*a)
