"""Binding of the paged key/value cache: block tables and slot maps, and the
attention over the pages (rules as in include/sdpa.h)."""
from __future__ import annotations

import functools

from . import _native
from .api import call_native


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
    of the table, entries) gets slots of -1 and keeps its length. The outputs that are
    not given share one allocation: while one of them is kept, all are."""
    return call_native("page_slots", stream, seqlens, (slots, positions, starts, seqlens_out, free_range_out), seqlens,
                       new_tokens, block_table, free_pages, free_range, page_size, rows, width, slots, positions,
                       starts, seqlens_out, free_range_out)


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
    The workspace (sdpa_fwd_paged_workspace_size bytes) is allocated when not given.
    Short sequences are 0.5 to 3 us faster under a table whose rows hold no more than
    512 keys."""
    return call_native("fwd_paged", stream, q, (out, lse), q, k_pages, v_pages, block_table, seqlens_k, scale, softcap,
                       window_left, out, lse, workspace)
