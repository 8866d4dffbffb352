"""Pools and tables that a server lays out in other ways: keys and values of a page side
by side in one pool, all layers' pools in one tensor, tables far wider than the
sequences."""
from __future__ import annotations

import math

import pytest
import torch

from paged_ref import check, make
from scaled_dot_product_06_gb300 import sdpa_fwd_paged, sdpa_qk_norm_rope

pytestmark = pytest.mark.gpu


def pools(x):
    """(name, keys, values): the pages of x as parts of larger tensors, on the GPU."""
    k, v = x["k_pages"].cuda(), x["v_pages"].cuda()
    n, h_kv, page, d = k.shape
    junk = float("nan")
    both = torch.full((n, 2, h_kv, page, d), junk, dtype=k.dtype, device="cuda")
    both[:, 0], both[:, 1] = k, v
    yield "side by side", both[:, 0], both[:, 1]
    rows = torch.full((n, page, 2, h_kv, d), junk, dtype=k.dtype, device="cuda")
    rows[:, :, 0], rows[:, :, 1] = k.transpose(1, 2), v.transpose(1, 2)
    yield "a token's side by side", rows[:, :, 0].transpose(1, 2), rows[:, :, 1].transpose(1, 2)
    layers = torch.full((n, 3, 2, h_kv, page, d), junk, dtype=k.dtype, device="cuda")
    layers[:, 1, 0], layers[:, 1, 1] = k, v
    yield "a page of all layers", layers[:, 1, 0], layers[:, 1, 1]
    heads = torch.full((h_kv, n, page, d + 8), junk, dtype=k.dtype, device="cuda")
    heads[..., :d] = k.transpose(0, 1)
    yield "a head's pages, padded rows", heads[..., :d].transpose(0, 1), v


@pytest.mark.parametrize("d,t", [(64, torch.float16), (128, torch.bfloat16)], ids=str)
def test_parts_of_larger_pools(d, t):
    x = make(3, 8, 2, 1, [300, 1, 777], 16, d, d, t, seed=d)
    rest = {n: x[n].cuda() for n in ("q", "block_table", "seqlens_k")}
    want = sdpa_fwd_paged(k_pages=x["k_pages"].cuda(), v_pages=x["v_pages"].cuda(), **rest)
    check(x, want, 1 / math.sqrt(d))
    k, v = (torch.randn(3, 1, 2, d, generator=torch.Generator().manual_seed(1)).to(t).cuda() for _ in range(2))
    slots = torch.tensor([[5], [3 * 16 + 2], [-1]], dtype=torch.int32, device="cuda")
    for name, kp, vp in pools(x):
        got = sdpa_fwd_paged(k_pages=kp, v_pages=vp, **rest)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), name
        if kp.shape[-1] == d and kp.stride(2) % 8 == 0:
            k_was, v_was = kp.clone(), vp.clone()
            sdpa_qk_norm_rope(rest["q"].transpose(1, 2), k, None, None, v=v, kv_slots=slots, k_out=kp, v_out=vp)
            for was, new, now in ((k_was, k, kp), (v_was, v, vp)):
                was[0, :, 5], was[3, :, 2] = new[0, 0], new[1, 0]
                assert torch.equal(now.nan_to_num(7.0), was.nan_to_num(7.0)), name


@pytest.mark.parametrize("b,longest", [(1, 17), (3, 512), (10, 1000), (80, 300)])
def test_tables_wider_than_the_sequences(b, longest):
    """The same short sequences under tables that leave them whole and that cut them."""
    lens = [(longest * (5 * i + 2)) // 7 % longest for i in range(b - 1)] + [longest]
    x = make(b, 8, 2, 1, lens, 16, 64, 64, torch.bfloat16, seed=b)
    for wide in (0, 1 << 13, 1 << 17):
        table = torch.full((b, max(wide // 16, x["block_table"].shape[1])), -1, dtype=torch.int32)
        table[:, :x["block_table"].shape[1]] = x["block_table"]
        y = dict(x, block_table=table)
        for left in (-1, 200):
            got = sdpa_fwd_paged(**{n: t.cuda() for n, t in y.items()}, window_left=left)
            check(x, got, 1 / 8, left=left)
