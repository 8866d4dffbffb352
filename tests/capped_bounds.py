"""Element-wise error bounds of attention with capped scores, from its roundings.

With u = finfo(dtype).eps / 2 (one rounding to the io type), |.| element-wise:

* The capped score is off by at most e_s = softcap * 2^-20 plus the fp32 dot
  product's error; cap_r8 states softcap * 2^-21, the other half is left for
  the fp32 sum of the exact 16-bit products (d <= 192 terms: relative error
  below d * 2^-24 of sum|q k|, a term of its own here). P is then off by
  2 e_s relative (its own score and the row's sum), plus 2^-20 for the
  exponentials and the sum.
* O: P rounded once (u), the product summed in fp32, O rounded once:
  |dO_err| <= (u + e_p) P|V| + u |O|.
* dV: the same with P^T|dO|.
* D = sum dO * O uses the rounded O: off by e_D = sum |dO| * (error of O).
* dS = P (dP - D)(1 - tanh^2): off by u |dS| (rounded once) + e_p |dS| +
  (1 - tanh^2) P e_D, and where the cap bends the score's own error moves
  1 - tanh^2 by 2 e_s / softcap of P |dP - D|; dQ and dK sum that against |K|
  and |Q| and round once.
* fp16 loses relative precision below 2^-14, where its numbers lie 2^-24 apart:
  every rounded P or dS may be off by 2^-25 absolute (P by that times 256, the
  largest stale factor of the running maximum, over a row sum of at least 1),
  and so may every rounded output (an output of 3e-5 is rounded by up to 3e-8,
  which is 2^-10 of it and not the 2^-11 of u).
* fp32 accumulation: 2^-16 of the sums of absolute values covers up to 256
  partial sums of 2^-24 each.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle
from oracle import sdpa_oracle as so


def u_of(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def head_bounds(pr, b, h, q, k, v, do, dtype):
    """(o, lse, dq, dk, dv) references of one head and their bounds."""
    u, acc = u_of(dtype), 2.0 ** -16
    sub = 2.0 ** -25 if dtype == torch.float16 else 0.0
    hk = pr.kv_head(h)
    q_h, k_h, v_h, do_h = (so._f64(x[b, i]) for x, i in ((q, h), (k, hk), (v, hk), (do, h)))
    rows, cols = np.arange(pr.S_q), np.arange(pr.S_kv)
    s = so.scores(pr, q_h, k_h, None, rows, cols)
    seen = np.isfinite(s)
    p, lse = so.softmax_rows(s)
    z = so.dropout_scale(pr, b, h, rows, cols)
    pz = p * z
    # error of a score: cap_r8's and the fp32 dot product's
    dot = abs(pr.scale) * (np.abs(q_h) @ np.abs(k_h).T) * pr.D_qk * 2.0 ** -24
    e_s = np.where(seen, (pr.softcap * 2.0 ** -20 if pr.softcap else 0.0) + dot, 0.0).max(
        axis=1, initial=0.0)[:, None]
    e_p = 2 * e_s + 2.0 ** -20
    o = pz @ v_h
    o_err = ((u + e_p + acc) * pz + 256 * sub * seen) @ np.abs(v_h) + u * np.abs(o) + sub
    lse_err = e_s[:, 0] + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)) + pr.softcap)
    dv = pz.T @ do_h
    dv_err = ((u + e_p + acc) * pz + sub * seen).T @ np.abs(do_h) + u * np.abs(dv) + sub
    dp = do_h @ v_h.T
    dd = (do_h * o).sum(1, keepdims=True)
    dd_err = (np.abs(do_h) * o_err).sum(1, keepdims=True) + acc * (np.abs(do_h) * np.abs(o)).sum(
        1, keepdims=True)
    t = np.where(seen, s, 0.0) / pr.softcap if pr.softcap else np.zeros_like(p)
    fac = 1.0 - t * t
    raw = p * (dp * z - dd)
    ds = raw * fac
    bend = 2 * e_s / pr.softcap * np.abs(raw) if pr.softcap else 0.0
    dp_err = acc * (np.abs(do_h) @ np.abs(v_h).T) * z
    ds_err = (u + e_p) * np.abs(ds) + bend + fac * p * (dd_err + dp_err) + sub * seen
    sc = abs(pr.scale)
    dq, dk = pr.scale * ds @ k_h, pr.scale * ds.T @ q_h
    dq_err = sc * (ds_err + acc * np.abs(ds)) @ np.abs(k_h) + u * np.abs(dq) + sub
    dk_err = sc * (ds_err + acc * np.abs(ds)).T @ np.abs(q_h) + u * np.abs(dk) + sub
    return (o, lse, dq, dk, dv), (o_err, lse_err, dq_err, dk_err, dv_err)


def bounds(pr, q, k, v, do, dtype):
    """References (o, lse, dq, dk, dv) of a batch-mode problem and their bounds."""
    shapes = [(pr.B, pr.H, pr.S_q, pr.D_v), (pr.B, pr.H, pr.S_q), (pr.B, pr.H, pr.S_q, pr.D_qk),
              (pr.B, pr.kv_heads, pr.S_kv, pr.D_qk), (pr.B, pr.kv_heads, pr.S_kv, pr.D_v)]
    ref, err = [np.zeros(x) for x in shapes], [np.zeros(x) for x in shapes]
    u = u_of(dtype)
    for b in range(pr.B):
        for h in range(pr.H):
            r, e = head_bounds(pr, b, h, q, k, v, do, dtype)
            for i, at in enumerate((h, h, h, pr.kv_head(h), pr.kv_head(h))):
                # dK and dV sum over the heads of a group in fp32 and round once
                ref[i][b, at] += r[i]
                err[i][b, at] += e[i] + (u * np.abs(r[i]) if i > 2 else 0.0)
    return ref, err


def assert_within(name, got, ref, err):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    ninf = np.isneginf(ref)
    assert np.array_equal(np.isneginf(got), ninf), f"{name}: -inf places differ"
    assert np.all(np.isfinite(got[~ninf])), f"{name}: non-finite values"
    over = np.abs(got[~ninf] - ref[~ninf]) - err[~ninf] - 1e-30
    assert over.size == 0 or over.max() <= 0, (
        f"{name}: {int((over > 0).sum())} of {over.size} elements past their bound, worst by "
        f"{over.max():.3e}")
