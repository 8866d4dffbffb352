"""Refusals of the block tables and slot maps and of the append into pages, on the
CPU before any CUDA call, and the plain form the GPU tests compare with."""
import ctypes

import pytest
import torch

from paged_ref import page_slots
from scaled_dot_product_06_gb300 import _native, sdpa_page_slots, sdpa_qk_norm_rope
from test_abi import MIS, NULL, P, lib  # noqa: F401

BAD, UNS, ALIGN, OK = (_native.SDPA_ERR_INVALID_ARG, _native.SDPA_ERR_UNSUPPORTED, _native.SDPA_ERR_MISALIGNED,
                       _native.SDPA_OK)
ODD = ctypes.c_void_p((1 << 20) + 2)


def slots(lib, b=2, page=16, wide=10, stride=10, pool=30, rows=0, width=1, lens=P, new=P, table=P, ring=P, span=P,
          to=P, pos=P, starts=NULL, lens_out=P, span_out=P):
    return lib.sdpa_page_slots(b, page, wide, stride, pool, rows, width, lens, new, table, ring, span, to, pos,
                               starts, lens_out, span_out, None)


def test_refusals(lib):  # noqa: F811
    for kw in (dict(b=-1), dict(page=0), dict(wide=-1), dict(pool=-1), dict(rows=-1, width=0), dict(width=-2),
               dict(rows=4, width=1), dict(rows=4, width=0), dict(starts=P), dict(stride=9), dict(lens=NULL),
               dict(new=NULL), dict(table=NULL), dict(ring=NULL), dict(span=NULL), dict(to=NULL), dict(pos=NULL),
               dict(lens_out=NULL), dict(span_out=NULL)):
        assert slots(lib, **kw) == BAD, kw
    for kw in (dict(b=1 << 31), dict(page=1 << 31, pool=1), dict(pool=1 << 27), dict(wide=1 << 28, stride=1 << 28),
               dict(rows=1 << 31, width=0, starts=P), dict(b=1 << 20, width=1 << 12), dict(b=1 << 20, wide=2048, stride=2048),
               dict(stride=1 << 50)):
        assert slots(lib, **kw) == UNS, kw
    for kw in (dict(to=ODD), dict(pos=MIS), dict(lens=ctypes.c_void_p((1 << 20) + 1)), dict(span=ODD),
               dict(span_out=ODD), dict(table=ctypes.c_void_p((1 << 20) + 3))):
        assert slots(lib, **kw) == ALIGN, kw


def rows_of(ptr=1 << 20, st=(1 << 16, 512, 64)):
    return ctypes.byref(_native.Rows(ptr, *st))


def append(lib, b=2, s=3, n_pages=4, page=16, slots=P, k_out=None, v_out=None):
    r = rows_of()
    return lib.sdpa_qk_norm_rope_paged(b, s, 4, 2, 64, 64, 0, r, r, r, r, k_out or r, v_out or r, 0, 0, NULL, NULL,
                                       0, NULL, NULL, NULL, 0, 1e-6, slots, n_pages, page, None)


def test_append_refusals(lib):  # noqa: F811
    assert append(lib, n_pages=-1) == BAD and append(lib, page=0) == BAD and append(lib, slots=NULL) == BAD
    assert append(lib, n_pages=1 << 20, page=1 << 20) == UNS and append(lib, page=1 << 40) == UNS
    assert append(lib, slots=ODD) == ALIGN
    assert append(lib, k_out=rows_of(st=(1 << 16, 512, 63))) == ALIGN
    assert append(lib, v_out=rows_of(ptr=(1 << 20) + 4)) == ALIGN
    assert append(lib, k_out=rows_of(ptr=None)) == BAD
    # the page stride of a single page is not looked at, nor are no pages
    assert append(lib, b=0, slots=NULL) == OK
    assert append(lib, s=0) == OK


def test_binding_refusals():
    n = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sdpa_page_slots(n, n, n.view(2, 1), n, n, 16, width=1)
    q = torch.zeros(1, 1, 2, 64).half()
    with pytest.raises(ValueError, match="CUDA"):
        sdpa_qk_norm_rope(q, q, None, None, kv_slots=n)


def test_plain_form():
    """By hand: pages of 4; request 0 grows inside its page, 1 takes two pages, 2 has
    ended, 3 asks for more pages than are left, 4 needs none."""
    table = [[7, -1, -1], [-1, -1, -1], [3, 5, -1], [2, -1, -1], [6, -1, -1]]
    ring = [9, 1, 0, 4, 8, 10, 11, 12, 13, 14, 15, 16]
    got = page_slots([2, 0, 5, 4, 1], [1, 6, -1, 5, 2], table, ring, [12, 15], 4, width=6)
    s, p, starts, lens, span, t, r = got
    assert starts is None and lens == [3, 6, 0, 4, 3] and span == [14, 17]
    assert s[:6] == [30] + [-1] * 5 and p[:6] == [2] + [0] * 5
    assert s[6:12] == [36, 37, 38, 39, 4, 5] and p[6:12] == [0, 1, 2, 3, 4, 5]
    assert s[12:18] == [-1] * 6 and s[18:24] == [-1] * 6 and p[18:24] == [4, 5, 6, 7, 8, 0]
    assert s[24:30] == [25, 26, -1, -1, -1, -1]
    assert t[1] == [9, 1, -1] and t[3] == [2, -1, -1] and r[3:5] == [3, 5]
    packed = page_slots([2, 0, 5, 4, 1], [1, 6, -1, 5, 2], table, ring, [12, 15], 4, rows=16)
    assert packed[0] == [30, 36, 37, 38, 39, 4, 5, -1, -1, -1, -1, -1, 25, 26, -1, -1]
    assert packed[2] == [0, 1, 7, 7, 12, 14]
    # the last request's tokens have no entries any more
    cut = page_slots([2, 0, 5, 4, 1], [1, 6, -1, 5, 2], table, ring, [12, 18], 4, rows=13)
    assert cut[2] == [0, 1, 7, 7, 12, 13] and cut[3] == [3, 6, 0, 9, 1] and cut[0][12] == -1 and cut[1][12] == 1
