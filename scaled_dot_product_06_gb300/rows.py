"""Binding of the calls around the attention: the norm and rotation of queries
and keys (names and rules as in include/sdpa.h).

As in ``api``, the functions check tensor properties, allocate outputs with
torch and pass pointers and strides; all arithmetic is in libsdpa.so.
"""
from __future__ import annotations

import functools
import struct

import torch

from . import _native
from .api import _DTYPE_CODE, _ptr, _run, _stream_ptr, call_native, check_workspace, new_tensor

_pack_rows = struct.Struct("Pqqq").pack  # the bytes of an sdpa_rows_t


def check_rows(name, t, shape, dtype, device):
    """The strides of a 4-D tensor with contiguous rows, of this type, shape and device."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on the device of q")
    strides = t.stride()
    if strides[3] != 1 and t.numel():
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return strides


def check_flat(name, t, shape, dtype, device):
    """The pointer of a contiguous tensor of this type, shape and device."""
    if t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on the device of q")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _token_rows(name, t, shape, dtype, device):
    """sdpa_rows_t of a [batch, token, head, width] input."""
    sb, st, sh, _ = check_rows(name, t, shape, dtype, device)
    return _pack_rows(t.data_ptr(), sb, st, sh)


def _head_rows(name, t, shape, dtype, device):
    """sdpa_rows_t of a [batch, head, row, width] input."""
    sb, sh, st, _ = check_rows(name, t, shape, dtype, device)
    return _pack_rows(t.data_ptr(), sb, st, sh)


def _check_output(name, t):
    strides = t.stride()
    if 0 in strides and any(st == 0 and n > 1 for n, st in zip(t.shape, strides)):
        raise ValueError(f"{name} must not be an expanded tensor")


def _table(dev, cos, sin, positions, b, s):
    """(rot, pointers of cos and sin, n_pos, pointer of positions)."""
    if cos is None or sin is None:
        if cos is not sin:
            raise ValueError("cos and sin go together")
        return 0, None, None, 0, None
    if cos.dim() != 2:
        raise ValueError("cos and sin must have shape (n_pos, rot / 2)")
    shape = cos.shape
    pc = check_flat("cos", cos, shape, torch.float32, dev)
    ps = check_flat("sin", sin, shape, torch.float32, dev)
    pp = None if positions is None else check_flat("positions", positions, (b, s), torch.int32, dev)
    return 2 * shape[1], pc, ps, shape[0], pp


def _weights(dt, dev, q_weight, k_weight, d):
    """(pointers, 1 when they are fp32 or 0 when they have q's type)."""
    w = q_weight if q_weight is not None else k_weight
    if w is None:
        return None, None, 0
    wt = w.dtype
    if wt != torch.float32 and wt != dt:
        raise ValueError("the weights must both be fp32 or both have q's dtype")
    pq = None if q_weight is None else check_flat("q_weight", q_weight, (d,), wt, dev)
    pk = None if k_weight is None else check_flat("k_weight", k_weight, (d,), wt, dev)
    return pq, pk, int(wt == torch.float32)


def _check_qkv(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or (v is not None and v.dim() != 4):
        raise ValueError("q, k and v must have 4 dimensions")
    if q.dtype not in _DTYPE_CODE:
        raise ValueError("q, k, v must be bf16 or fp16")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")


def sdpa_qk_norm_rope(q, k, cos, sin, *, v=None, positions=None, q_weight=None, k_weight=None,
                      eps=1e-6, interleaved=False, kv_rows=None, kv_slots=None, q_out=None, k_out=None,
                      v_out=None, stream=None):
    """Root-mean-square norm of each query and key head, and its rotation by
    position, from the projection's layout to the attention's in one pass.

    q [b, s, h, d], k [b, s, h_kv, d] and optionally v [b, s, h_kv, d_v] may be
    slices of one fused projection (any strides that are multiples of 16
    bytes). Returns (q_out [b, h, s, d], k_out [b, h_kv, s, d], v_out or None).
    cos, sin (fp32 [n_pos, rot / 2], None: no rotation) hold the angles of the
    first rot = 2 cos.shape[1] elements of a head, paired (i, i + rot / 2) or,
    with interleaved, (2 i, 2 i + 1); positions (int32 [b, s]) picks each
    token's row, by default its place in the sequence. q_weight, k_weight [d]
    (both fp32 or both of q's dtype) scale the normalised heads; None leaves
    that side unnormalised. kv_rows (int32 [b]) makes k_out and v_out caches
    [b, h_kv, rows, d] that get token t of sequence i in row kv_rows[i] + t
    (tokens outside the cache are dropped, no other row is touched).
    kv_slots (int32 [b, s]) makes them the pages [n_pages, h_kv, page_size, d] of
    a paged cache instead: each token goes to row slot % page_size of page
    slot // page_size, or nowhere where the slot is outside the pages (see
    sdpa_page_slots)."""
    return call_native("qk_norm_rope", stream, q, (q_out, k_out, v_out), q, k, cos, sin, v, positions, q_weight,
                       k_weight, eps, interleaved, kv_rows, kv_slots, q_out, k_out, v_out)


@functools.lru_cache(maxsize=256)
def _bwd_bytes(b, s, h, h_kv, d, d_v) -> int:
    return int(_native.lib().sdpa_qk_norm_rope_bwd_workspace_size(b, s, h, h_kv, d, d_v))


def sdpa_qk_norm_rope_bwd_workspace_size(b, s, h, h_kv, d, d_v) -> int:
    """Workspace bytes of sdpa_qk_norm_rope_bwd with a weight."""
    return _bwd_bytes(int(b), int(s), int(h), int(h_kv), int(d), int(d_v))


def sdpa_qk_norm_rope_bwd(dq_out, dk_out, q, k, cos, sin, *, dv_out=None, positions=None,
                          q_weight=None, k_weight=None, eps=1e-6, interleaved=False, dq=None, dk=None,
                          dv=None, dq_weight=None, dk_weight=None, workspace=None, stream=None):
    """Backward of sdpa_qk_norm_rope (without caches). dq_out [b, h, s, d],
    dk_out [b, h_kv, s, d] and optionally dv_out are the gradients of its
    outputs, q and k its inputs. Returns (dq [b, s, h, d], dk, dv or None,
    dq_weight or None, dk_weight or None); dq, dk, dv may be given as slices of
    one fused gradient. The weight gradients have the weights' dtype and, for
    the same call, the same bits in every run (their sums' order depends on the
    sizes and on which of values and weights there are)."""
    _check_qkv(q, k, None)
    if dq_out.dim() != 4 or dk_out.dim() != 4 or (dv_out is not None and dv_out.dim() != 4):
        raise ValueError("dq_out, dk_out and dv_out must have 4 dimensions")
    b, s, h, d = q.shape
    h_kv, dt, dev = k.shape[2], q.dtype, q.device
    d_v = d if dv_out is None else dv_out.shape[3]
    if dv is not None and dv_out is None:
        raise ValueError("dv without dv_out")
    q_in = _token_rows("q", q, (b, s, h, d), dt, dev)
    k_in = _token_rows("k", k, (b, s, h_kv, d), dt, dev)
    gq = _head_rows("dq_out", dq_out, (b, h, s, d), dt, dev)
    gk = _head_rows("dk_out", dk_out, (b, h_kv, s, d), dt, dev)
    gv = None if dv_out is None else _head_rows("dv_out", dv_out, (b, h_kv, s, d_v), dt, dev)
    rot, cos_p, sin_p, n_pos, pos_p = _table(dev, cos, sin, positions, b, s)
    qw_p, kw_p, fp32 = _weights(dt, dev, q_weight, k_weight, d)
    if dq is None:
        dq = new_tensor((b, s, h, d), dt, dev, stream)
    if dk is None:
        dk = new_tensor((b, s, h_kv, d), dt, dev, stream)
    if dv is None and dv_out is not None:
        dv = new_tensor((b, s, h_kv, d_v), dt, dev, stream)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        if t is not None:
            _check_output(name, t)
    q_to = _token_rows("dq", dq, (b, s, h, d), dt, dev)
    k_to = _token_rows("dk", dk, (b, s, h_kv, d), dt, dev)
    v_to = None if dv is None else _token_rows("dv", dv, (b, s, h_kv, d_v), dt, dev)
    grads = []
    for name, w, g in (("dq_weight", q_weight, dq_weight), ("dk_weight", k_weight, dk_weight)):
        if w is None:
            if g is not None:
                raise ValueError(f"{name} without its weight")
        elif g is None:
            g = new_tensor((d,), w.dtype, dev, stream)
        else:
            check_flat(name, g, (d,), w.dtype, dev)
        grads.append(g)
    if workspace is None and (q_weight is not None or k_weight is not None):
        workspace = new_tensor(max(_bwd_bytes(b, s, h, h_kv, d, d_v), 1), torch.uint8, dev, stream, scratch=True)
    ws = (None, 0) if workspace is None else check_workspace(workspace, dev)
    _run(q, "sdpa_qk_norm_rope_bwd", b, s, h, h_kv, d, d_v, _DTYPE_CODE[dt], gq, gk, gv, q_in, k_in, q_to,
         k_to, v_to, rot, int(bool(interleaved)), cos_p, sin_p, n_pos, pos_p, qw_p, kw_p, fp32, eps,
         _ptr(grads[0]), _ptr(grads[1]), *ws, _stream_ptr(stream, q))
    return dq, dk, dv, grads[0], grads[1]
