"""Binding of the paged key/value cache: block tables and slot maps, and the
attention over the pages (rules as in include/sdpa.h)."""
from __future__ import annotations

import functools

import torch

from . import _native
from .api import _DTYPE_CODE, _run, _stream_ptr, check_workspace, new_tensor
from .rows import _pack_rows, check_flat


def _check_table(block_table, b, index):
    """(width, stride) of a block table [b, width] with contiguous rows, on device `index`."""
    shape, (stride, inner) = block_table.shape, block_table.stride() if block_table.dim() == 2 else (0, 0)
    if len(shape) != 2 or shape[0] != b or block_table.dtype is not torch.int32 \
            or block_table.get_device() != index:
        raise ValueError(f"block_table must be an int32 tensor of {b} rows on the other tensors' device")
    width = shape[1]
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
    i32, index = torch.int32, seqlens.get_device()
    if seqlens.dim() != 1 or free_pages.dim() != 1:
        raise ValueError("seqlens and free_pages must have one dimension")
    one = seqlens.shape
    b, n_pages = one[0], free_pages.shape[0]
    n_p = _flat("seqlens", seqlens, one, i32, index)
    x_p = _flat("new_tokens", new_tokens, one, i32, index)
    f_p = _flat("free_pages", free_pages, (n_pages,), i32, index)
    r_p = _flat("free_range", free_range, (2,), torch.int64, index)
    table_width, stride = _check_table(block_table, b, index)
    dev = seqlens.device
    if rows is not None:
        shape, r, w = (rows,), rows, 0
        if starts is None:
            starts = new_tensor((b + 1,), i32, dev, stream)
            s_p = starts.data_ptr()
        else:
            s_p = _flat("starts", starts, (b + 1,), i32, index)
    elif starts is None:
        shape, r, w, s_p = (b, width), 0, width, None
    else:
        raise ValueError("starts are of packed rows")
    if slots is None:
        slots = new_tensor(shape, i32, dev, stream)
        o_p = slots.data_ptr()
    else:
        o_p = _flat("slots", slots, shape, i32, index)
    if positions is None:
        positions = _like(slots, stream)
        p_p = positions.data_ptr()
    else:
        p_p = _flat("positions", positions, shape, i32, index)
    if seqlens_out is None:
        seqlens_out = _like(seqlens, stream)
        l_p = seqlens_out.data_ptr()
    else:
        l_p = _flat("seqlens_out", seqlens_out, one, i32, index)
    if free_range_out is None:
        free_range_out = _like(free_range, stream)
        e_p = free_range_out.data_ptr()
    else:
        e_p = _flat("free_range_out", free_range_out, (2,), torch.int64, index)
    _run(seqlens, "sdpa_page_slots", b, page_size, table_width, stride, n_pages, r, w, n_p, x_p,
         block_table.data_ptr(), f_p, r_p, o_p, p_p, s_p, l_p, e_p, _stream_ptr(stream, seqlens))
    return slots, positions, starts, seqlens_out, free_range_out


def _like(t, stream):
    """A new tensor as t (a little cheaper than by its shape)."""
    return torch.empty_like(t) if stream is None else new_tensor(t.shape, t.dtype, t.device, stream)


def _flat(name, t, shape, dtype, index):
    if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on the device of seqlens")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _pages(name, t, shape, dtype, index):
    """The bytes of an sdpa_rows_t of pages [n_pages, h_kv, page_size, d]."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on the device of q")
    sp, sh, sr, sd = t.stride()
    if sd != 1 and t.numel():
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return _pack_rows(t.data_ptr(), sp, sr, sh)


@functools.lru_cache(maxsize=256)
def _bytes(h, h_kv, s_q, d_qk, d_v, page_size, table_width) -> int:
    return int(_native.lib().sdpa_fwd_paged_workspace_size(h, h_kv, s_q, d_qk, d_v, page_size, table_width))


def sdpa_fwd_paged_workspace_size(h, h_kv, s_q, d_qk, d_v, page_size, table_width) -> int:
    """Workspace bytes of sdpa_fwd_paged, for any batch and lengths (0: it needs none)."""
    return _bytes(int(h), int(h_kv), int(s_q), int(d_qk), int(d_v), int(page_size), int(table_width))


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
    one, pool, vals = q.shape, k_pages.shape, v_pages.shape
    if len(one) != 4 or len(pool) != 4 or len(vals) != 4:
        raise ValueError("q, k_pages and v_pages must have 4 dimensions")
    dt = q.dtype
    code = _DTYPE_CODE.get(dt)
    if code is None:
        raise ValueError("q, k_pages, v_pages must be bf16 or fp16")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    index = q.get_device()
    b, h, s_q, d_qk = one
    n_pages, h_kv, page, _ = pool
    d_v = vals[3]
    k_in = _pages("k_pages", k_pages, (n_pages, h_kv, page, d_qk), dt, index)
    v_in = _pages("v_pages", v_pages, (n_pages, h_kv, page, d_v), dt, index)
    if seqlens_k.dtype is not torch.int32 or seqlens_k.get_device() != index or not seqlens_k.is_contiguous() \
            or seqlens_k.shape != (b,):
        raise ValueError(f"seqlens_k must be a contiguous int32 tensor of {b} elements on the device of q")
    table_width, stride = _check_table(block_table, b, index)
    dev = q.device
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
    if workspace is not None:
        ws = check_workspace(workspace, dev)
    else:
        need = _bytes(h, h_kv, s_q, d_qk, d_v, page, table_width)
        if need:
            workspace = new_tensor((need,), torch.uint8, dev, stream, scratch=True)
        ws = workspace.data_ptr() if need else None, need
    _run(q, "sdpa_fwd_paged", b, h, h_kv, s_q, d_qk, d_v, d_qk ** -0.5 if scale is None else scale, softcap or 0.0,
         -1 if window_left is None else window_left, code, q.data_ptr(), k_in, v_in, n_pages, page,
         block_table.data_ptr(), table_width, stride, seqlens_k.data_ptr(), o_p, l_p, *ws, _stream_ptr(stream, q))
    return out, lse
