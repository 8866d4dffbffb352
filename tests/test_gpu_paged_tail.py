"""Many keys of little weight each behind one of most, in the attention over a paged
cache: what they add up to is in O as it is in LSE."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from capped_bounds import u_of
from paged_ref import f64
from scaled_dot_product_06_gb300 import sdpa_device_error, sdpa_fwd_paged
from scaled_dot_product_06_gb300.inputs import DTYPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [8, 64])
def test_the_tail_of_a_long_row(t, rows):
    """Two keys have nearly all weight, each of 131070 others 2^-25.4 of one of them, 2^-9.4
    in all: as many sequences as SMs, so that none is cut and a warpgroup sums half of
    them, behind one of the two. In the first half of the columns the two keys' values are
    0, in the second they are 1.

    A sum of n keys in fp32 adds n / 16 times, each cut off at 2^-23 of it; a thread adds a
    key's P to its sum n / 256 times, to 2^-24. (Weights of 2^-25.4 rounded to fp16 are 0.)"""
    n, b, d, page = 131072, 152, 64, 64
    dt = DTYPES[t]
    g = torch.Generator().manual_seed(5)
    k, v = torch.zeros(n, d), torch.randint(8, 25, (n, d), generator=g) / 16
    two = [7, 135]
    k[two, 0] = 8.8125                     # 16 k / 8 = 17.625 = 25.43 log(2)
    v[two, :d // 2], v[two, d // 2:] = 0.0, 1.0
    q = torch.zeros(b, rows, 1, d)
    q[..., 0] = 16.0
    pages = n // page
    x = {"q": q.to(dt), "k_pages": k.view(pages, 1, page, d).to(dt), "v_pages": v.view(pages, 1, page, d).to(dt),
         "block_table": torch.arange(pages, dtype=torch.int32).expand(b, pages).contiguous(),
         "seqlens_k": torch.full((b,), n, dtype=torch.int32)}
    o, lse = sdpa_fwd_paged(**{name: t.cuda() for name, t in x.items()})
    torch.cuda.synchronize()
    assert sdpa_device_error() == 0
    s = np.zeros(n)
    s[two] = 17.625
    w = np.exp(s - 17.625)
    total = w.sum()
    want = w @ v.double().numpy() / total
    err = (2.0 ** -23 * n / 16 + 2.0 ** -19 + u_of(dt)) * np.abs(want)
    assert (want[:d // 2] < 2.0 ** -9).all() and (err[:d // 2] < 2.0 ** -16).all()
    assert (np.abs(f64(o) - want) <= err).all()
    assert (np.abs(f64(lse) - 17.625 - np.log(total)) <= 2.0 ** -18 + 2.0 ** -24 * n / 256).all()
    assert torch.equal(o, o[:1, :1].expand(o.shape))
