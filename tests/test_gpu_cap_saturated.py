"""Gradients of capped attention where every score of a row lies at the cap, above
or below: 1 - tanh^2 is small there, and has to be so to a small relative error.

Bound of dS = P (dP - D) f, f = 1 - tanh^2 = 4 e / (1 + e)^2 with e = exp(2 x), x =
S' / cap: f moves by at most the relative error of e, which is twice that of x
(the dot product's d 2^-24 sum|q k| |scale| / cap, and a few roundings of 2^-24 of
the exponent: |x| 2^-21 covers them), 2^-22 of the exponential and fewer than 20
roundings of r and f: 2^-19 in all. Scores up to 4.1 caps (12 / (2 log2 e)) may take f
as 4 r (1 - r), off by 2^-21 of r and so by up to 2^-9 more below. P is good to 2 cap
2^-20 + 2^-20, dS is rounded once (u), D uses the rounded O.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from capped_bounds import u_of
from scaled_dot_product_06_gb300 import sdpa_bwd, sdpa_device_error, sdpa_fwd
from scaled_dot_product_06_gb300.inputs import DTYPES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("at", [-10.0, -6.0, -4.0, -3.0, 4.0, 6.0, 10.0])
@pytest.mark.parametrize("d,d_v", [(64, 64), (128, 128), (192, 128)])
def test_gradients_at_the_cap(d, d_v, at, deterministic):
    s_q, s_kv, cap, dt = 128, 192, 1.0, DTYPES["bf16"]
    u, acc = u_of(dt), 2.0 ** -16
    g = torch.Generator().manual_seed(d)
    scale = 1.0 / np.sqrt(d)
    q = torch.randn(1, 1, s_q, d, generator=g) * 0.25
    k = torch.randn(1, 1, s_kv, d, generator=g) * 0.25
    root = (abs(at) * cap / scale) ** 0.5
    q[..., 0], k[..., 0] = root, root * np.sign(at)
    q, k = q.to(dt), k.to(dt)
    v, do = (torch.randn(1, 1, s, d_v, generator=g).to(dt) for s in (s_kv, s_q))
    gq, gk, gv, gdo = (t.cuda() for t in (q, k, v, do))
    kw = dict(scale=float(scale), softcap=cap)
    o, lse = sdpa_fwd(gq, gk, gv, **kw)
    dq, dk, _, _ = sdpa_bwd(gq, gk, gv, o, gdo, lse, deterministic=deterministic, **kw)
    torch.cuda.synchronize()
    assert sdpa_device_error() == 0

    q, k, v, do = (t[0, 0].double().numpy() for t in (q, k, v, do))
    x = scale * (q @ k.T) / cap
    f = 1.0 / np.cosh(x) ** 2
    assert np.abs(x - at).max() < 0.7
    p = np.exp(cap * np.tanh(x))
    p /= p.sum(1, keepdims=True)
    e_p = 2 * cap * 2.0 ** -20 + 2.0 ** -20
    o64 = p @ v
    o_err = (u + e_p + acc) * (p @ np.abs(v)) + u * np.abs(o64)
    dp, dd = do @ v.T, (do * o64).sum(1, keepdims=True)
    dd_err = (np.abs(do) * (o_err + acc * np.abs(o64))).sum(1, keepdims=True)
    ds = p * (dp - dd) * f
    e_f = 2 * d * 2.0 ** -24 * scale * (np.abs(q) @ np.abs(k).T) / cap + np.abs(x) * 2.0 ** -21 + 2.0 ** -19
    e_f = e_f + np.where(np.abs(x) < 4.2, 2.0 ** -9, 0.0)
    ds_err = (u + e_p + e_f + acc) * np.abs(ds) + f * p * (dd_err + acc * (np.abs(do) @ np.abs(v).T))
    for name, got, ref, err in (("dq", dq, ds @ k, ds_err @ np.abs(k)), ("dk", dk, ds.T @ q, ds_err.T @ np.abs(q))):
        err = scale * err + u * np.abs(scale * ref)
        off = np.abs(got[0, 0].double().cpu().numpy() - scale * ref)
        assert (off <= err).all(), (name, float((off / err).max()))
        # (the bound says something: the largest values are far above theirs)
        assert (np.abs(scale * ref) > 4 * err).any(), name
