"""Capped-score entry points on the CPU: argument errors before any CUDA call,
the oracle's cap against differences, and the reciprocal form of the cap."""
import ctypes

import numpy as np
import pytest

import oracle
from scaled_dot_product_06_gb300 import _native
from test_abi import MIS, NULL, P, lib  # noqa: F401


def fwd(lib, cap=30.0, scale=0.125, left=-1, right=0, br=0, keep=NULL, rec=NULL, p=0.0, dqk=64, dv=64,
        h=2, h_kv=2, skv=128, q=P, lse=P):
    return lib.sdpa_fwd_capped(1, h, h_kv, 128, skv, dqk, dv, scale, cap, left, right, br, keep, rec, p,
                               0, 0, 0, q, P, P, P, lse, None)


def bwd(lib, cap=30.0, phases=7, scale=0.125, ws=P, nbytes=1 << 30, dq=P):
    return lib.sdpa_bwd_phases_capped(phases, 1, 2, 2, 128, 128, 64, 64, scale, cap, -1, 0, 0, NULL, 0.0,
                                      0, 0, 0, P, P, P, P, P, P, dq, P, P, ws, nbytes, None)


def test_argument_errors(lib):  # noqa: F811
    bad = _native.SDPA_ERR_INVALID_ARG
    for cap in (0.0, -1.0, float("nan"), float("inf"), 4097.0):
        assert fwd(lib, cap=cap) == bad
        assert bwd(lib, cap=cap) == bad
    assert fwd(lib, cap=1e-38, scale=1e3) == bad
    assert fwd(lib, scale=float("nan")) == bad
    assert fwd(lib, h_kv=3) == bad
    assert fwd(lib, q=NULL) == bad
    assert fwd(lib, lse=MIS) == _native.SDPA_ERR_MISALIGNED
    assert fwd(lib, dqk=96) == _native.SDPA_ERR_UNSUPPORTED
    assert fwd(lib, p=0.1, rec=P, keep=P) == bad
    assert fwd(lib, p=0.1, skv=132, rec=P) == _native.SDPA_ERR_UNSUPPORTED
    assert fwd(lib, skv=0, q=NULL) == _native.SDPA_OK
    assert bwd(lib, phases=0) == bad
    assert bwd(lib, ws=NULL) == _native.SDPA_ERR_WORKSPACE
    assert bwd(lib, nbytes=64) == _native.SDPA_ERR_WORKSPACE
    assert bwd(lib, dq=NULL) == bad
    for f, extra in ((lib.sdpa_fwd_varlen_capped, 0),):
        st = f(2, 2, 2, 128, 128, 64, 64, 64, 64, 0.125, 30.0, -1, 0, 0, NULL, NULL, 0.0, 0, 0, 0, NULL,
               P, P, P, P, P, P, None)
        assert st == bad
    st = lib.sdpa_bwd_phases_varlen_capped(7, 2, 2, 2, 128, 128, 64, 64, 64, 64, 0.125, -2.0, -1, 0, 0,
                                           NULL, 0.0, 0, 0, 0, P, P, P, P, P, P, P, P, P, P, P, P,
                                           1 << 30, None)
    assert st == bad


@pytest.mark.parametrize("cap", [0.5, 3.0, 50.0])
def test_oracle_cap_against_differences(cap):
    pr = oracle.Problem(1, 1, 6, 9, 4, 4, 0.7, window=(-1, 2), softcap=cap)
    rng = np.random.default_rng(0)
    x = {n: rng.standard_normal((1, 1, s, 4)) * 2 for n, s in
         (("q", 6), ("k", 9), ("v", 9), ("do", 6))}
    g = dict(zip(("q", "k", "v"), oracle.backward(pr, x["q"], x["k"], x["v"], x["do"])[:3]))
    for n in g:
        for _ in range(5):
            d = rng.standard_normal(x[n].shape)
            val = []
            for sgn in (1, -1):
                y = dict(x)
                y[n] = x[n] + sgn * 1e-6 * d
                val.append((oracle.forward(pr, y["q"], y["k"], y["v"])[0] * x["do"]).sum())
            assert abs((val[0] - val[1]) / 2e-6 - (g[n] * d).sum()) < 1e-7


def test_reciprocal_form_of_the_cap():
    """cap - 2 cap r with four values sharing one reciprocal, in fp32: within
    the documented cap * 2^-21 for any mix of saturated and small scores."""
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.standard_normal(4000) * s for s in (1e-3, 1.0, 30.0, 1e3, 1e30)])
    x = rng.permutation(x).astype(np.float32).reshape(-1, 4)
    f = np.float32
    for cap in (0.01, 30.0, 4096.0):
        c = f(2 * 1.4426950408889634 * 0.1 / cap)
        with np.errstate(over="ignore"):
            y = np.minimum(x * c, f(30))
        a = f(1) + np.exp2(y.astype(np.float64)).astype(f)
        p01, p23 = a[:, 0] * a[:, 1], a[:, 2] * a[:, 3]
        assert np.isfinite(p01 * p23).all()
        inv = f(1) / (p01 * p23)
        i01, i23 = inv * p23, inv * p01
        r = np.stack([i01 * a[:, 1], i01 * a[:, 0], i23 * a[:, 3], i23 * a[:, 2]], 1)
        got = cap - 2 * cap * r.astype(np.float64)
        ref = cap * np.tanh(x.astype(np.float64) * 0.1 / cap)
        assert np.abs(got - ref).max() <= cap * 2.0 ** -21
