"""Values that are not a number in sdpa_fwd_prefix: a visible key or a query that
is none makes exactly the rows that see it none (O and LSE), whatever parts the
keys were cut into; every other row keeps its bits.
"""
from __future__ import annotations

import pytest
import torch

from scaled_dot_product_06_gb300 import sdpa_device_error, sdpa_fwd_prefix
from scaled_dot_product_06_gb300.inputs import DTYPES

pytestmark = pytest.mark.gpu

NAN = float("nan")

# (b, h, h_kv, s_q, s_prefix, s_max, lens, d, d_v, dtype)
CASES = [
    (3, 8, 2, 1, 700, 300, [1, 130, 300], 128, 128, "bf16"),       # a quarter of the own keys a warp
    (2, 33, 1, 1, 300, 300, [300, 97], 64, 64, "fp16"),            # R = 33: both warpgroups the same rows
    (2, 16, 1, 9, 400, 500, [9, 444], 128, 128, "bf16"),           # R = 144: two row tiles
    (2, 4, 4, 4, 513, 260, [4, 259], 192, 128, "fp16"),            # drafted tokens, wide heads
    (1, 8, 8, 1, 40000, 20, [20], 64, 64, "bf16"),                 # many parts of the prefix
    (5, 10, 2, 1, 0, 9000, [9000, 1, 4097, 8999, 128], 128, 128, "bf16"),  # many of the own keys
    (180, 4, 1, 1, 300, 500, [(37 * i) % 500 + 1 for i in range(180)], 64, 64, "bf16"),  # items on demand
]


def case_id(c):
    return f"b{c[0]}h{c[1]}kv{c[2]}q{c[3]}-p{c[4]}-own{c[5]}-d{c[7]}-{c[9]}"


def make(c, seed=3):
    b, h, h_kv, s_q, s_p, s_max, lens, d, d_v, dt = c
    g = torch.Generator().manual_seed(seed)

    def r(*shape, mul=1.0):
        return (torch.randn(*shape, generator=g) * mul).to(DTYPES[dt]).cuda()

    return {"q": r(b, h, s_q, d, mul=2.0), "k_prefix": r(h_kv, s_p, d), "v_prefix": r(h_kv, s_p, d_v),
            "k": r(b, h_kv, s_max, d), "v": r(b, h_kv, s_max, d_v),
            "seqlens_k": torch.tensor(lens, dtype=torch.int32).cuda()}


def expect(x, clean, hit, cap, **kw):
    """hit [b, h, s_q]: the rows that have to be NaN. Capped, a visible score shares
    the roundings of one reciprocal with hidden ones: rows of a hit head keep their
    bits only up to the cap's own error, twice cap 2^-20 and the log-sum's 2^-20."""
    o, lse = sdpa_fwd_prefix(**x, softcap=cap, **kw)
    torch.cuda.synchronize()
    assert sdpa_device_error() == 0
    hit = hit.cuda()
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.isfinite(o[~hit].float()).all() and torch.isfinite(lse[~hit]).all()
    if cap:
        assert ((lse - clean[1])[~hit].abs() <= 2 * (2 * cap + 1 + clean[1][~hit].abs()) * 2.0 ** -20).all()
        heads = ~hit.any(2)
        assert torch.equal(o[heads], clean[0][heads]) and torch.equal(lse[heads], clean[1][heads])
    else:
        assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("c", CASES, ids=case_id)
def test_reaches_the_rows_that_see_it(c, cap):
    b, h, h_kv, s_q, s_p, s_max, lens = c[:7]
    group = h // h_kv
    x = make(c)
    clean = sdpa_fwd_prefix(**x, softcap=cap)
    assert torch.isfinite(clean[0].float()).all()
    none = torch.zeros(b, h, s_q, dtype=torch.bool)
    # a key of the prefix: first, in the middle, last
    for j in sorted({0, s_p // 2, s_p - 1}) if s_p else ():
        y = dict(x, k_prefix=x["k_prefix"].clone())
        y["k_prefix"][h_kv - 1, j, 5] = NAN
        hit = none.clone()
        hit[:, (h_kv - 1) * group:] = True
        expect(y, clean, hit, cap)
    # a key of the last sequence's own
    n = lens[-1]
    for j in sorted({0, n // 2, n - 1}):
        y = dict(x, k=x["k"].clone())
        y["k"][b - 1, 0, j] = NAN
        hit = none.clone()
        for t in range(s_q):
            hit[b - 1, :group, t] = j <= n - s_q + t
        expect(y, clean, hit, cap)
    # a query
    y = dict(x, q=x["q"].clone())
    y["q"][0, h - 1, s_q - 1, 0] = NAN
    hit = none.clone()
    hit[0, h - 1, s_q - 1] = True
    expect(y, clean, hit, cap)


@pytest.mark.parametrize("scale", [0.1, -0.1])
def test_infinite_scores(scale):
    """A key that is infinite in one element: rows with a score of +inf are NaN (as
    inf - inf is), rows with -inf give it no weight."""
    x = make((2, 8, 2, 1, 300, 200, [200, 77], 64, 64, "bf16"))
    clean = sdpa_fwd_prefix(**x, scale=scale)
    kp = x["k_prefix"].clone()
    kp[0, 100, 7] = float("inf")
    o, lse = sdpa_fwd_prefix(**dict(x, k_prefix=kp), scale=scale)
    up = (x["q"][:, :, :, 7].float() * scale > 0)
    up[:, 4:] = False
    assert torch.isnan(o[up]).all() and torch.isnan(lse[up]).all()
    assert torch.isfinite(o[~up].float()).all() and torch.isfinite(lse[~up]).all()
    assert torch.equal(o[:, 4:], clean[0][:, 4:])
