"""What lies behind a sequence's last key decides nothing in sdpa_fwd_prefix, with
capped scores either: the same bits with NaN, infinities, large and small numbers
and zeros there.
"""
from __future__ import annotations

import pytest
import torch

from scaled_dot_product_06_gb300 import sdpa_device_error, sdpa_fwd_prefix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h,s_q", [(8, 1), (8, 3), (66, 1), (32, 9)])
@pytest.mark.parametrize("d,d_v", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_same_bits(d, d_v, h, s_q, cap):
    b, h_kv, s_p, s_max = 12, 2, 200, 400
    g = torch.Generator().manual_seed(d + s_q)
    lens = [s_q, 127, 128, 129, 131, 37, 38, 39, 40, 399, 400, 257]

    def r(*shape, mul=1.0):
        return (torch.randn(*shape, generator=g) * mul).bfloat16().cuda()

    q, kp, vp = r(b, h, s_q, d, mul=3.0), r(h_kv, s_p, d), r(h_kv, s_p, d_v)
    k, v = r(b, h_kv, s_max, d), r(b, h_kv, s_max, d_v)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    behind = (torch.arange(s_max, device="cuda") >= n[:, None])[:, None, :, None]
    want = None
    for fill in (0.0, 1e-3, 5.0, -300.0, 1e30, float("inf"), float("nan")):
        kk, vv = k.masked_fill(behind, fill), v.masked_fill(behind, fill)
        got = sdpa_fwd_prefix(q, kp, vp, kk, vv, n, softcap=cap)
        torch.cuda.synchronize()
        assert torch.isfinite(got[0].float()).all()
        want = want or got
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), fill
    assert sdpa_device_error() == 0
