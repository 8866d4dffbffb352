"""Refusals of the norm-and-rotation calls, on the CPU: the C entry points
before any CUDA call, the binding on tensors it must not pass on."""
import ctypes

import pytest
import torch

from scaled_dot_product_06_gb300 import _native, sdpa_qk_norm_rope, sdpa_qk_norm_rope_bwd
from test_abi import MIS, NULL, P, lib  # noqa: F401

BAD, UNS, ALIGN, WS = (_native.SDPA_ERR_INVALID_ARG, _native.SDPA_ERR_UNSUPPORTED,
                       _native.SDPA_ERR_MISALIGNED, _native.SDPA_ERR_WORKSPACE)


def rows(ptr=1 << 20, sb=1 << 16, sr=1 << 10, sh=128):
    return ctypes.byref(_native.Rows(ptr, sb, sr, sh))


USUAL = object()


def fwd(lib, b=2, s=8, h=4, h_kv=2, d=128, d_v=128, dtype=0, q=USUAL, k=USUAL, v=NULL, q_out=USUAL, k_out=USUAL,
        v_out=NULL, rot=64, cos=P, sin=P, n_pos=64, pos=NULL, qw=P, kw=P, eps=1e-6, kv_rows=NULL, cache=0):
    q, k, q_out, k_out = (rows() if x is USUAL else x for x in (q, k, q_out, k_out))
    return lib.sdpa_qk_norm_rope(b, s, h, h_kv, d, d_v, dtype, q, k, v, q_out, k_out, v_out, rot, 0, cos, sin,
                                 n_pos, pos, qw, kw, 1, eps, kv_rows, cache, None)


def bwd(lib, b=2, s=8, d=128, dqw=P, dkw=P, ws=P, nbytes=1 << 30, qw=P, kw=P, dv_out=NULL, dv=NULL, q=USUAL,
        dq=USUAL):
    q, dq = (rows() if x is USUAL else x for x in (q, dq))
    return lib.sdpa_qk_norm_rope_bwd(b, s, 4, 2, d, d, 0, rows(), rows(), dv_out, q, rows(), dq, rows(), dv, 64,
                                     0, P, P, 64, NULL, qw, kw, 1, 1e-6, dqw, dkw, ws, nbytes, None)


def test_forward_refusals(lib):  # noqa: F811
    assert fwd(lib, b=-1) == BAD
    assert fwd(lib, h=0) == BAD
    assert fwd(lib, dtype=5) == UNS
    assert fwd(lib, d=96) == UNS
    assert fwd(lib, d=64, d_v=128) == UNS
    for rot in (8, 144, -16, 24):
        assert fwd(lib, rot=rot) == UNS
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert fwd(lib, eps=eps) == BAD
    assert fwd(lib, cos=NULL) == BAD
    assert fwd(lib, sin=MIS) == ALIGN
    assert fwd(lib, n_pos=7) == BAD  # fewer angles than tokens, no positions
    assert fwd(lib, pos=ctypes.c_void_p((1 << 20) + 2)) == ALIGN
    assert fwd(lib, qw=MIS) == ALIGN
    assert fwd(lib, q=NULL) == BAD
    assert fwd(lib, q=rows(ptr=(1 << 20) + 8)) == ALIGN
    assert fwd(lib, k=rows(sr=1028)) == ALIGN
    assert fwd(lib, q_out=rows(sh=12)) == ALIGN
    assert fwd(lib, v=rows()) == BAD
    assert fwd(lib, v_out=rows()) == BAD
    assert fwd(lib, kv_rows=MIS, cache=-1) == BAD
    assert fwd(lib, b=1 << 20, s=1 << 20) == UNS
    # nothing to do: no pointer is looked at
    assert fwd(lib, s=0, q=NULL, cos=NULL) == _native.SDPA_OK
    assert fwd(lib, b=0, k_out=NULL) == _native.SDPA_OK


def test_backward_refusals(lib):  # noqa: F811
    assert bwd(lib, dqw=NULL) == BAD
    assert bwd(lib, kw=NULL) == BAD
    assert bwd(lib, dv=rows()) == BAD
    assert bwd(lib, dv_out=rows()) == BAD
    assert bwd(lib, d=80) == UNS
    assert bwd(lib, q=NULL) == BAD
    assert bwd(lib, dq=rows(sb=3)) == ALIGN
    assert bwd(lib, dqw=MIS) == ALIGN
    assert bwd(lib, ws=NULL) == WS
    assert bwd(lib, nbytes=16) == WS
    assert bwd(lib, ws=ctypes.c_void_p((1 << 20) + 16)) == ALIGN
    size = lib.sdpa_qk_norm_rope_bwd_workspace_size
    assert size(2, 8, 4, 2, 128, 128) % 256 == 0 and size(2, 8, 4, 2, 128, 128) > 0
    assert size(1, 1 << 20, 32, 8, 128, 128) <= (4 * 152 + 3) * 128 * 4 + 256
    assert size(2, 8, 4, 2, 96, 96) == 0
    assert size(0, 8, 4, 2, 128, 128) == 0


def test_binding_refusals():
    q, k = torch.zeros(1, 4, 2, 64).half(), torch.zeros(1, 4, 2, 64).half()
    with pytest.raises(ValueError):
        sdpa_qk_norm_rope(q, k, None, None)  # not CUDA tensors
    with pytest.raises(ValueError):
        sdpa_qk_norm_rope(q[0], k, None, None)
    with pytest.raises(ValueError):
        sdpa_qk_norm_rope(q.float(), k.float(), None, None)
    with pytest.raises(ValueError):
        sdpa_qk_norm_rope_bwd(q, k, q, k[0], None, None)
