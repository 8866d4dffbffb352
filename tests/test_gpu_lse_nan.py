"""The forward's statistics of rows that see something that is not a number: O and
LSE are none there (-inf is left to rows that see no key), with dropout too.
"""
from __future__ import annotations

import pytest
import torch

from scaled_dot_product_06_gb300 import sdpa_bwd, sdpa_device_error, sdpa_fwd
from scaled_dot_product_06_gb300.inputs import Shape, make_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p", [0.0, 0.5])
@pytest.mark.parametrize("cap", [None, 20.0])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_it(d, cap, p):
    x = make_inputs(Shape(1, 2, 300, 260, d, d, 2), "bf16")
    q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "do"))
    k[:, 0, 101] = float("nan")
    q[:, 1, 77, 3] = float("nan")
    # row i sees keys up to i - 40: the first 40 rows see none
    kw = dict(window=(-1, 0), bottom_right=True, softcap=cap)
    o, lse = sdpa_fwd(q, k, v, dropout_p=p, seed=1, offset=2, **kw)
    torch.cuda.synchronize()
    assert sdpa_device_error() == 0
    sees = torch.zeros(2, 300, dtype=torch.bool)
    sees[0, 101 + 40:] = True
    sees[1, 77] = True
    empty = torch.zeros(2, 300, dtype=torch.bool)
    empty[:, :40] = True
    sees, empty = sees.cuda(), empty.cuda()
    assert torch.isnan(o[0][sees]).all() and torch.isnan(lse[0][sees]).all()
    assert torch.isneginf(lse[0][empty]).all() and not o[0][empty].any()
    rest = ~sees & ~empty
    assert torch.isfinite(o[0][rest].float()).all() and torch.isfinite(lse[0][rest]).all()
    if p:
        return
    # P of such a row is none, and so is dV of the keys it sees
    dq, _, dv, _ = sdpa_bwd(q, k, v, o, do, lse, **kw)
    assert torch.isnan(dq[0][sees]).all()
    assert torch.isnan(dv[0, 0]).all() and torch.isnan(dv[0, 1, :38]).all()
