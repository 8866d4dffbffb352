"""Attention with capped scores (softcap) against the fp64 oracle, element by
element within bounds derived from its roundings (capped_bounds), in batch and
packed mode; equalities between its forms; capture into a graph.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from capped_bounds import assert_within, bounds
from oracle import varlen as ovl
from scaled_dot_product_06_gb300 import (SDPA_BWD_DKDV, SDPA_BWD_DQ, SDPA_BWD_PREPROCESS, sdpa_bwd,
                                         sdpa_bwd_phases, sdpa_bwd_varlen, sdpa_bwd_workspace_size,
                                         sdpa_device_error, sdpa_dropout_mask, sdpa_fwd, sdpa_fwd_varlen)
from scaled_dot_product_06_gb300.inputs import (DTYPES, Shape, make_inputs, make_packed_inputs,
                                                seqstarts)

pytestmark = pytest.mark.gpu

SEED, OFFSET = 0x51, 3

# (B, H, H_kv, S_q, S_kv, D_qk, D_v, dtype, softcap, factor on q, window, bottom_right, p)
CASES = [
    (1, 2, 2, 256, 256, 128, 128, "bf16", 50.0, 4.0, (-1, 0), False, 0.0),    # causal
    (2, 2, 2, 200, 333, 64, 64, "fp16", 30.0, 4.0, (-1, -1), False, 0.0),     # ragged, no mask
    (1, 4, 2, 300, 300, 128, 128, "bf16", 5.0, 30.0, (-1, 0), False, 0.0),    # most scores at the cap
    (1, 2, 2, 160, 257, 192, 128, "bf16", 20.0, 4.0, (-1, 0), True, 0.0),     # d_qk = 192
    (1, 2, 1, 192, 192, 192, 128, "fp16", 20.0, 4.0, (70, 0), False, 0.1),    # window, dropout
    (1, 8, 1, 130, 260, 64, 64, "bf16", 10.0, 4.0, (-1, 0), False, 0.0),      # one K/V head: split dK/dV
    (1, 8, 1, 256, 128, 128, 128, "fp16", 10.0, 4.0, (-1, -1), False, 0.2),   # split, dropout
    (1, 2, 2, 300, 100, 128, 128, "bf16", 15.0, 4.0, (-1, 0), True, 0.0),     # rows that see no key
    (1, 2, 2, 200, 128, 64, 64, "bf16", 15.0, 4.0, (300, 0), False, 0.0),     # one key tile
    (1, 2, 2, 1, 640, 128, 128, "bf16", 50.0, 4.0, (-1, 0), True, 0.0),       # one query
    (1, 1, 1, 129, 385, 64, 64, "fp16", 4096.0, 2.0, (-1, -1), False, 0.0),   # the largest cap
    (1, 1, 1, 64, 96, 64, 64, "bf16", 0.01, 1.0, (-1, -1), False, 0.0),       # a cap that flattens
]


def case_id(c):
    B, H, H_kv, S_q, S_kv, D, _, dt, cap, f, win, br, p = c
    return f"b{B}h{H}kv{H_kv}-{S_q}x{S_kv}-d{D}-{dt}-cap{cap}-w{win[0]}_{win[1]}{'-br' * br}-p{p}"


def inputs(c):
    B, H, H_kv, S_q, S_kv, D_qk, D_v, dt, cap, f, win, br, p = c
    x = make_inputs(Shape(B, H, S_q, S_kv, D_qk, D_v, H_kv), dt)
    x["q"] = (x["q"].float() * f).to(DTYPES[dt])
    return x


def on_gpu(x):
    return tuple(x[n].cuda() for n in ("q", "k", "v", "do"))


def settled():
    torch.cuda.synchronize()
    assert sdpa_device_error() == 0


@pytest.mark.parametrize("scale_sign", [1.0, -1.0], ids=["", "negative"])
@pytest.mark.parametrize("c", CASES, ids=case_id)
def test_capped_matches_oracle(c, scale_sign):
    B, H, H_kv, S_q, S_kv, D_qk, D_v, dt, cap, f, win, br, p = c
    x = inputs(c)
    scale = scale_sign / np.sqrt(D_qk)
    pr = oracle.Problem(B, H, S_q, S_kv, D_qk, D_v, scale, False, p, SEED, OFFSET, H_kv, win, br,
                        softcap=cap)
    ref, err = bounds(pr, x["q"], x["k"], x["v"], x["do"], DTYPES[dt])
    q, k, v, do = on_gpu(x)
    kw = dict(scale=scale, dropout_p=p, seed=SEED, offset=OFFSET, window=win, bottom_right=br,
              softcap=cap)
    o, lse = sdpa_fwd(q, k, v, **kw)
    settled()
    assert_within("o", o, ref[0], err[0])
    assert_within("lse", lse, ref[1], err[1])
    for det in (False, True):
        dq, dk, dv, db = sdpa_bwd(q, k, v, o, do, lse, deterministic=det, **kw)
        settled()
        assert db is None
        for i, g in ((2, dq), (3, dk), (4, dv)):
            assert_within(f"{('dq', 'dk', 'dv')[i - 2]} deterministic={det}", g, ref[i], err[i])


@pytest.mark.parametrize("dt,D_qk,D_v,cap", [("bf16", 128, 128, 50.0), ("fp16", 64, 64, 8.0),
                                             ("bf16", 192, 128, 30.0)])
def test_packed_matches_oracle(dt, D_qk, D_v, cap):
    """Packed sequences of 1, 0, 300, 128 and 77 tokens, causal."""
    H, H_kv = 4, 2
    st = seqstarts([1, 0, 300, 128, 77])
    total = st[-1]
    x = make_packed_inputs(H, total, total, D_qk, D_v, dt, H_kv)
    x["q"] = (x["q"].float() * 4).to(DTYPES[dt])
    scale = 1.0 / np.sqrt(D_qk)
    pk = ovl.Packed(tuple(st), tuple(st), H, D_qk, D_v, scale, True, H_kv=H_kv, softcap=cap)
    q, k, v, do = on_gpu(x)
    starts = torch.tensor(st, dtype=torch.int32, device="cuda")
    kw = dict(scale=scale, is_causal=True, softcap=cap)
    o, lse = sdpa_fwd_varlen(q, k, v, starts, starts, 300, 300, **kw)
    grads = [sdpa_bwd_varlen(q, k, v, o, do, lse, starts, starts, 300, 300, deterministic=det, **kw)
             for det in (False, True)]
    settled()
    for i in range(pk.B):
        lo, hi = st[i], st[i + 1]
        if lo == hi:
            continue
        ref, err = bounds(pk.sequence(i), *(x[n][None, :, lo:hi] for n in ("q", "k", "v", "do")),
                          DTYPES[dt])
        got = [[o, lse, *g] for g in grads]
        for det in (0, 1):
            for j, name in enumerate(("o", "lse", "dq", "dk", "dv")):
                assert_within(f"{name} of sequence {i}, {det}", got[det][j][None, :, lo:hi], ref[j],
                              err[j])


def test_forms_agree():
    """is_causal and its window, phases one by one, recorded dropout bits and
    a wide cap beside no cap."""
    shp = Shape(2, 4, 256, 256, 128, 128, 2)
    q, k, v, do = on_gpu(make_inputs(shp, "bf16"))
    o, lse = sdpa_fwd(q, k, v, is_causal=True, softcap=20.0)
    o2, lse2 = sdpa_fwd(q, k, v, window=(-1, 0), softcap=20.0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    whole = sdpa_bwd(q, k, v, o, do, lse, is_causal=True, softcap=20.0, deterministic=True)
    # the same workspace room as the whole call's: it decides how dK/dV is split
    ws = torch.empty(sdpa_bwd_workspace_size(2, 4, 256, 256, 128, 128, 2, True), dtype=torch.uint8,
                     device="cuda")
    parts = [torch.empty_like(t) for t in (q, k, v)]
    for phase in (SDPA_BWD_PREPROCESS, SDPA_BWD_DKDV, SDPA_BWD_DQ):
        sdpa_bwd_phases(phase, q, k, v, o, do, lse, is_causal=True, softcap=20.0, deterministic=True,
                        workspace=ws, dq=parts[0], dk=parts[1], dv=parts[2])
    assert all(torch.equal(a, b) for a, b in zip(whole, parts))
    # dropout: bits drawn in the kernels, recorded by the forward, drawn beforehand
    kw = dict(is_causal=True, softcap=20.0, dropout_p=0.25, seed=9, offset=2)
    words = 2 * 4 * 256 * 256 // 32
    rec = torch.zeros(words, dtype=torch.int32, device="cuda")
    o, lse = sdpa_fwd(q, k, v, **kw)
    o2, _ = sdpa_fwd(q, k, v, dropout_mask_out=rec, **kw)
    mask = sdpa_dropout_mask(2, 4, 256, 256, 0.25, 9, 2)
    o3, _ = sdpa_fwd(q, k, v, dropout_mask=mask, **kw)
    assert torch.equal(o, o2) and torch.equal(o, o3)
    g = [sdpa_bwd(q, k, v, o, do, lse, deterministic=True, dropout_mask=m, **kw)
         for m in (None, rec, mask)]
    assert all(torch.equal(a, b) for a, b in zip(g[0][:3], g[1][:3]))
    assert all(torch.equal(a, b) for a, b in zip(g[0][:3], g[2][:3]))
    settled()
    # softcap 0 and None are the uncapped call
    a, b = sdpa_fwd(q, k, v, softcap=0.0)[0], sdpa_fwd(q, k, v)[0]
    assert torch.equal(a, b)


def test_captured_beside_eager():
    """A captured step, replayed on new inputs, gives the eager step's results
    (the deterministic backward, whose side stream joins the capture)."""
    shp = Shape(1, 4, 192, 192, 128, 128)
    kw = dict(is_causal=True, softcap=30.0)
    a, b = make_inputs(shp, "bf16"), make_inputs(shp, "bf16", seed_base=50)
    q, k, v, do = on_gpu(a)

    def step():
        o, lse = sdpa_fwd(q, k, v, **kw)
        return (o, lse, *sdpa_bwd(q, k, v, o, do, lse, deterministic=True, **kw)[:3])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (do, "do")):
        t.copy_(b[n])
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in out]
    assert all(torch.equal(x, y) for x, y in zip(got, step()))
    settled()


def test_gradients_against_differences():
    """<dX, dir> against a central difference of the fp64 oracle along dir: ties
    the formula's factor 1 - tanh^2 to the function, not to another formula."""
    shp = Shape(1, 1, 64, 64, 64, 64)
    x = make_inputs(shp, "fp16")
    x["q"] = (x["q"].float() * 4).half()
    pr = oracle.Problem(1, 1, 64, 64, 64, 64, 0.125, True, softcap=3.0)
    q, k, v, do = on_gpu(x)
    o, lse = sdpa_fwd(q, k, v, scale=0.125, is_causal=True, softcap=3.0)
    dq, dk, dv, _ = sdpa_bwd(q, k, v, o, do, lse, scale=0.125, is_causal=True, softcap=3.0)
    ref, err = bounds(pr, x["q"], x["k"], x["v"], x["do"], torch.float16)
    d64 = {n: x[n].double().numpy() for n in ("q", "k", "v", "do")}
    rng = np.random.default_rng(1)
    h = 1e-5
    for name, g, e in (("q", dq, err[2]), ("k", dk, err[3]), ("v", dv, err[4])):
        d = rng.standard_normal(d64[name].shape)
        val = []
        for sgn in (1, -1):
            y = dict(d64)
            y[name] = d64[name] + sgn * h * d
            val.append((oracle.forward(pr, y["q"], y["k"], y["v"])[0] * d64["do"]).sum())
        diff = (val[0] - val[1]) / (2 * h)
        got = (g.double().cpu().numpy() * d).sum()
        # the gradient's own bound along d, and the difference's O(h^2) (third
        # derivatives of order 10^2) and cancellation (10^3 * 2^-53 / h) terms
        assert abs(got - diff) <= (e * np.abs(d)).sum() + 1e-6, name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [(-1, 0), (40, 0)])
def test_not_a_number_stays_where_it_is(d, window):
    """A key that is not a number reaches the queries that see it, all of them,
    and no other; a query that is not a number only itself."""
    x = make_inputs(Shape(1, 2, 300, 300, d, d, 2), "bf16")
    q, k, v = (x[n].cuda() for n in ("q", "k", "v"))
    kw = dict(scale=d ** -0.5, window=window, softcap=20.0)
    o0, lse0 = sdpa_fwd(q, k, v, **kw)
    bad_k, bad_q = k.clone(), q.clone()
    bad_k[:, 0, 101] = float("nan")
    bad_q[:, 1, 77, 3] = float("nan")
    o, lse = sdpa_fwd(bad_q, bad_k, v, **kw)
    settled()
    sees = torch.zeros(2, 300, dtype=torch.bool)
    sees[0, 101:] = True
    if window[0] >= 0:
        sees[0, 101 + window[0] + 1:] = False
    sees[1, 77] = True
    sees = sees.cuda()
    assert torch.isnan(o[0][sees]).all()
    # Not bit for bit: a visible score shares its reciprocal's roundings with
    # hidden ones. A score is off by at most cap 2^-20 in each of the two calls,
    # and so is the log-sum (with its own 2^-20, as in capped_bounds); a P at the
    # border of a rounding may then round the other way, once in P and in O.
    cap = 20.0
    ok = (lse - lse0).abs() <= 2 * (cap + 1 + lse0.abs() + cap) * 2.0 ** -20
    assert ok[0][~sees].all()
    u = 2.0 ** -8
    ok = (o.float() - o0.float()).abs() <= u * (2 * o0.float().abs() + v.float().abs().max()) + 2 * cap * 2.0 ** -20
    assert ok[0][~sees].all()


def test_refusals():
    shp = Shape(1, 2, 64, 64, 64, 64)
    x = make_inputs(shp, "bf16", with_bias=True)
    q, k, v, _ = on_gpu(x)
    with pytest.raises(ValueError):
        sdpa_fwd(q, k, v, softcap=5.0, bias=x["bias"].cuda())
    with pytest.raises(ValueError):
        sdpa_fwd(q, k, v, softcap=5.0, alibi_slopes=torch.ones(2, device="cuda"))
    for bad in (-1.0, float("nan"), float("inf"), 5000.0):
        with pytest.raises(RuntimeError, match="softcap"):
            sdpa_fwd(q, k, v, softcap=bad)
    with pytest.raises(RuntimeError, match="finite"):
        sdpa_fwd(q, k, v, softcap=1e-38, scale=1e3)
