"""How far a capped score may be off, from the arithmetic that forms it (fp32, four
values to one reciprocal), with the two approximate functions at their worst: the
exponential off by 2^-22 relative either way, the reciprocal by one unit in the last
place either way. Bound: with all roundings r is off by five roundings of 2^-24, the
reciprocal's 2^-23 and (1 - r) of the exponential's 2^-22 and of the exponent's own
error, so cap - 2 cap r by cap (7 r + 4 r (1 - r)) 2^-23 + cap 2^-23 <= cap 2^-20.
"""
import numpy as np
import pytest

F = np.float32


def r_of(x, c, ex, rc, factor):
    """r (and 4 e r^2) of rows of four raw scores; ex, rc: relative errors of the functions."""
    with np.errstate(over="ignore"):
        if factor:
            y = (x.astype(np.float64) * c + 2).astype(F)  # one rounding, as an FMA
            e = (np.exp2(np.minimum(y, F(32)).astype(np.float64)) * (1 + ex)).astype(F)
            a = (e.astype(np.float64) * 0.25 + 1).astype(F)
        else:
            y = np.minimum(x * c, F(30))
            e = (np.exp2(y.astype(np.float64)) * (1 + ex)).astype(F)
            a = F(1) + e
    p01, p23 = a[:, 0] * a[:, 1], a[:, 2] * a[:, 3]
    inv = (1 / (p01 * p23).astype(np.float64) * (1 + rc)).astype(F)
    assert np.isfinite(inv).all()
    i01, i23 = inv * p23, inv * p01
    r = np.stack([i01 * a[:, 1], i01 * a[:, 0], i23 * a[:, 3], i23 * a[:, 2]], 1)
    return r, (e * r) * r


@pytest.mark.parametrize("factor", [False, True])
@pytest.mark.parametrize("cap", [0.01, 30.0, 4096.0])
def test_score_within_its_bound(cap, factor):
    rng = np.random.default_rng(5)
    x = np.concatenate([rng.standard_normal(20000) * cap * s * 10 for s in (1e-3, 0.3, 1.0, 3.0, 1e3)])
    x = rng.permutation(x).astype(F).reshape(-1, 4)
    c = F(2 * 1.4426950408889634 * 0.1 / cap)
    t = x.astype(np.float64) * 0.1 / cap
    worst = 0.0
    for ex in (-2.0 ** -22, 0.0, 2.0 ** -22):
        for rc in (-2.0 ** -23, 0.0, 2.0 ** -23):
            r, f = r_of(x, c, ex, rc, factor)
            worst = max(worst, np.abs(cap - 2 * cap * r.astype(np.float64) - cap * np.tanh(t)).max() / cap)
            if factor:
                # 4 e r^2 against 1 - tanh^2 where the hold at 30 is out of reach, in units
                # of 2^-24: the exponential 4, the exponent (up to 29, off by two
                # roundings, times ln 2) 40, twice r 14, two products: below 64
                near = np.abs(t) < 10
                true = 1 / np.cosh(t[near]) ** 2
                assert (np.abs(f[near] / true - 1) <= 2.0 ** -18).all()
    assert worst <= 2.0 ** -20
    assert worst > 2.0 ** -21  # (half of it is not a bound)
