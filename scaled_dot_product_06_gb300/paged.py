"""Binding of the paged key/value cache: block tables and slot maps, and the
attention over the pages (rules as in include/sdpa.h)."""
from __future__ import annotations

import functools
import math

import torch

from . import _native
from .api import _DTYPE_CODE, _ptr, _run, _stream_ptr, check_workspace, new_tensor
from .rows import _pack_rows, check_flat, check_rows


def _check_table(block_table, b, device):
    """(width, stride) of a block table [b, width] with contiguous rows."""
    if block_table.dim() != 2 or block_table.shape[0] != b or block_table.dtype != torch.int32 \
            or block_table.device != device:
        raise ValueError(f"block_table must be an int32 tensor of {b} rows on the other tensors' device")
    width = block_table.shape[1]
    stride, inner = block_table.stride()
    if width > 1 and inner != 1:
        raise ValueError("block_table: the entries of a row must be contiguous")
    if b > 1 and stride < width:
        raise ValueError("block_table: its rows must not overlap")
    return width, stride


def sdpa_page_slots(seqlens, new_tokens, block_table, free_pages, free_range, page_size, *, rows=None,
                    width=None, slots=None, positions=None, starts=None, seqlens_out=None,
                    free_range_out=None, stream=None):
    """Gives pages to the new tokens of a batch and builds their slots, in one launch.

    seqlens [b]: tokens of each request in the cache; new_tokens [b]: tokens to
    come (0: idle, negative: the request has ended). block_table [b, w] gets the new
    pages, taken from the ring free_pages [n_pages], whose entries free_range[0]
    <= i < free_range[1] (modulo n_pages) are free; the pages of ended requests are
    written behind its end. All int32, free_range int64 [2].

    Either rows (packed: the tokens of all requests one after another, in
    tensors of `rows` entries) or width (padded: [b, width]). Returns (slots,
    positions, starts, seqlens_out, free_range_out): the slot page * page_size
    + row of each token, -1 where there is none; its position; packed, the offsets
    [b + 1] that the packed calls take (else None); the new lengths, for
    sdpa_fwd_paged; the new ring. seqlens and free_range may be given as
    seqlens_out and free_range_out. A request for which there is no room (pages, width
    of the table, entries) gets slots of -1 and keeps its length."""
    if not seqlens.is_cuda:
        raise ValueError("seqlens must be a CUDA tensor")
    if (rows is None) == (width is None):
        raise ValueError("either rows (packed) or width (padded)")
    dev, i32 = seqlens.device, torch.int32
    if seqlens.dim() != 1 or free_pages.dim() != 1:
        raise ValueError("seqlens and free_pages must have one dimension")
    b, n_pages = seqlens.shape[0], free_pages.shape[0]
    n_p = _flat("seqlens", seqlens, (b,), i32, dev)
    x_p = _flat("new_tokens", new_tokens, (b,), i32, dev)
    f_p = _flat("free_pages", free_pages, (n_pages,), i32, dev)
    r_p = _flat("free_range", free_range, (2,), torch.int64, dev)
    table_width, stride = _check_table(block_table, b, dev)
    packed = rows is not None
    if not packed and starts is not None:
        raise ValueError("starts are of packed rows")
    shape = (rows,) if packed else (b, width)
    made = []
    for name, t, sh, dt in (("slots", slots, shape, i32), ("positions", positions, shape, i32),
                            ("seqlens_out", seqlens_out, (b,), i32),
                            ("free_range_out", free_range_out, (2,), torch.int64),
                            ("starts", starts, (b + 1,) if packed else None, i32)):
        if t is not None:
            _flat(name, t, sh, dt, dev)
        elif sh is not None:
            t = new_tensor(sh, dt, dev, stream)
        made.append(t)
    slots, positions, seqlens_out, free_range_out, starts = made
    _run(seqlens, "sdpa_page_slots", b, page_size, table_width, stride, n_pages, rows if packed else 0,
         0 if packed else width, n_p, x_p, block_table.data_ptr(), f_p, r_p, slots.data_ptr(),
         positions.data_ptr(), _ptr(starts), seqlens_out.data_ptr(), free_range_out.data_ptr(),
         _stream_ptr(stream, seqlens))
    return slots, positions, starts, seqlens_out, free_range_out


def _flat(name, t, shape, dtype, device):
    if t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on the device of seqlens")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


@functools.lru_cache(maxsize=256)
def _bytes(h, h_kv, s_q, d_qk, d_v) -> int:
    return int(_native.lib().sdpa_fwd_paged_workspace_size(h, h_kv, s_q, d_qk, d_v))


def sdpa_fwd_paged_workspace_size(h, h_kv, s_q, d_qk, d_v) -> int:
    """Workspace bytes of sdpa_fwd_paged (for any batch, lengths and pages)."""
    return _bytes(int(h), int(h_kv), int(s_q), int(d_qk), int(d_v))


def sdpa_fwd_paged(q, k_pages, v_pages, block_table, seqlens_k, *, scale=None, softcap=None, window_left=None,
                   out=None, lse=None, workspace=None, stream=None):
    """Attention of each sequence's newest tokens over a paged cache. Returns
    (o [b, h, s_q, d_v], lse fp32 [b, h, s_q]).

    q [b, h, s_q, d_qk]; k_pages, v_pages [n_pages, h_kv, page_size, d] (any strides
    with contiguous rows, so pages kept as [n_pages, page_size, h_kv, d] come as
    their transpose(1, 2)); page_size a power of two from 8. block_table int32
    [b, w]: the pages of each sequence in order; seqlens_k int32 [b]: its keys,
    the s_q new tokens' among them (appended beforehand). New token t sees keys up to
    its own place seqlens_k - s_q + t, the last window_left + 1 of them if that is
    given. What the pages hold besides is not looked at. softcap as in sdpa_fwd.
    The workspace (sdpa_fwd_paged_workspace_size bytes) is allocated when not given."""
    if q.dim() != 4 or k_pages.dim() != 4 or v_pages.dim() != 4:
        raise ValueError("q, k_pages and v_pages must have 4 dimensions")
    dt, dev = q.dtype, q.device
    if dt not in _DTYPE_CODE:
        raise ValueError("q, k_pages, v_pages must be bf16 or fp16")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    b, h, s_q, d_qk = q.shape
    n_pages, h_kv, page, _ = k_pages.shape
    d_v = v_pages.shape[3]
    q_p = check_flat("q", q, (b, h, s_q, d_qk), dt, dev)
    sp, sh, sr, _ = check_rows("k_pages", k_pages, (n_pages, h_kv, page, d_qk), dt, dev)
    k_in = _pack_rows(k_pages.data_ptr(), sp, sr, sh)
    sp, sh, sr, _ = check_rows("v_pages", v_pages, (n_pages, h_kv, page, d_v), dt, dev)
    v_in = _pack_rows(v_pages.data_ptr(), sp, sr, sh)
    n_p = check_flat("seqlens_k", seqlens_k, (b,), torch.int32, dev)
    table_width, stride = _check_table(block_table, b, dev)
    if out is None:
        out = new_tensor((b, h, s_q, d_v), dt, dev, stream)
        o_p = out.data_ptr()
    else:
        o_p = check_flat("out", out, (b, h, s_q, d_v), dt, dev)
    if lse is None:
        lse = new_tensor((b, h, s_q), torch.float32, dev, stream)
        l_p = lse.data_ptr()
    else:
        l_p = check_flat("lse", lse, (b, h, s_q), torch.float32, dev)
    if workspace is None:
        need = _bytes(h, h_kv, s_q, d_qk, d_v)
        workspace = new_tensor(max(need, 1), torch.uint8, dev, stream, scratch=True)
        ws = workspace.data_ptr(), need
    else:
        ws = check_workspace(workspace, dev)
    _run(q, "sdpa_fwd_paged", b, h, h_kv, s_q, d_qk, d_v, 1.0 / math.sqrt(d_qk) if scale is None else scale,
         softcap or 0.0, -1 if window_left is None else window_left, _DTYPE_CODE[dt], q_p, k_in, v_in, n_pages,
         page, block_table.data_ptr(), table_width, stride, n_p, o_p, l_p, *ws, _stream_ptr(stream, q))
    return out, lse
