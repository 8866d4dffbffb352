"""Norm and rotation of queries and keys (sdpa_qk_norm_rope and its backward)
against plain fp64 arithmetic.

Bounds, element by element (u = finfo(dtype).eps / 2, one rounding of an
output; fp16 outputs below 2^-14 are rounded by up to 2^-25): everything else
is fp32. A row's mean of squares is a sum of at most 192 terms, 8 in a lane and
the rest in a tree, relative error below 16 * 2^-24; its rsqrt, the products
with x and w and the turn add less than 8 roundings of 2^-24 and the rsqrt's
2 ulp: 2^-18 of the sums of absolute values covers them. A weight gradient is
a sum over n rows, at most `chain` of them in one thread and 32 + 16 + 5 after
that, so (chain + 80) * 2^-24 of the sum of absolute values covers it and the
terms' own errors.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from scaled_dot_product_06_gb300 import (sdpa_bwd, sdpa_device_error, sdpa_fwd, sdpa_qk_norm_rope,
                                         sdpa_qk_norm_rope_bwd, sdpa_qk_norm_rope_bwd_workspace_size)
from scaled_dot_product_06_gb300.inputs import DTYPES

pytestmark = pytest.mark.gpu

EPS = 1e-6


def angles(n_pos, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * inv
    return a.cos().float(), a.sin().float()


def turn(x, c, s, rot, inter):
    """x [..., d] fp64 turned, and the same with absolute values (its bound's scale)."""
    half = rot // 2
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
    y, m = x.clone(), x.abs()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    m[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
    m[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, m


def reference(x, w, c, s, rot, inter):
    """[b, n, heads, d] fp64 -> attention's layout, and the bound's scale."""
    if w is not None:
        x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
    y, m = turn(x, c, s, rot, inter)
    return y.transpose(1, 2), m.transpose(1, 2)


def check(name, got, ref, scale, dtype):
    u = torch.finfo(dtype).eps / 2
    sub = 2.0 ** -25 if dtype == torch.float16 else 0.0
    got = got.double().cpu()
    assert got.shape == ref.shape, name
    assert torch.isfinite(got).all(), name
    over = (got - ref).abs() - (u * ref.abs() + 2.0 ** -18 * scale + sub)
    assert over.numel() == 0 or over.max() <= 0, f"{name}: past its bound by {over.max():.3e}"


# (b, s, h, h_kv, d, d_v, dtype, rot, interleaved, weight type, positions)
CASES = [
    (2, 37, 4, 2, 128, 128, "bf16", 128, False, "fp32", True),
    (1, 1, 1, 1, 64, 64, "fp16", 64, False, "io", False),
    (3, 5, 3, 1, 192, 128, "fp16", 64, True, "fp32", True),
    (1, 130, 5, 3, 192, 192, "bf16", 192, False, "io", True),
    (2, 9, 7, 7, 64, 64, "bf16", 16, False, "fp32", True),
    (2, 9, 2, 5, 128, 64, "bf16", 48, True, "fp32", True),
    (4, 17, 8, 2, 128, 128, "fp16", 96, False, None, True),    # rotation alone
    (2, 33, 4, 4, 128, 128, "bf16", 0, False, "fp32", False),  # norm alone
    (1, 1200, 16, 4, 128, 128, "bf16", 128, False, "fp32", True),  # four heads a group
    (1, 1300, 13, 3, 64, 64, "fp16", 32, True, "io", True),        # four heads a group, ragged
    (1, 700, 30, 6, 192, 128, "bf16", 64, False, "fp32", True),    # four heads a group
]


def case_id(c):
    return "b%d-s%d-h%d-kv%d-d%dx%d-%s-rot%d-i%d-%s-%d" % c


def make(c):
    b, s, h, h_kv, d, d_v, dt, rot, inter, wt, with_pos = c
    g = torch.Generator().manual_seed(sum(c[:6]))
    t = DTYPES[dt]
    qkv = (torch.randn(b, s, h * d + h_kv * (d + d_v), generator=g) * 2).to(t)
    x = {"qkv": qkv, "w": None, "pos": None}
    if wt:
        wdt = torch.float32 if wt == "fp32" else t
        x["w"] = [(1 + 0.2 * torch.randn(d, generator=g)).to(wdt) for _ in range(2)]
    n_pos = 5000
    if with_pos:
        x["pos"] = torch.randint(0, n_pos, (b, s), generator=g).to(torch.int32)
    x["cos"], x["sin"] = angles(n_pos, rot) if rot else (None, None)
    return x


def split(qkv, c):
    b, s, h, h_kv, d, d_v = c[:6]
    return (qkv[..., :h * d].unflatten(-1, (h, d)),
            qkv[..., h * d:(h + h_kv) * d].unflatten(-1, (h_kv, d)),
            qkv[..., (h + h_kv) * d:].unflatten(-1, (h_kv, d_v)))


def turns_of(x, c):
    b, s = c[:2]
    rot = c[7]
    if not rot:
        return torch.ones(b, s, 1, 0, dtype=torch.float64), torch.zeros(b, s, 1, 0, dtype=torch.float64)
    pos = x["pos"].long() if x["pos"] is not None else torch.arange(s).expand(b, s)
    return x["cos"].double()[pos][:, :, None], x["sin"].double()[pos][:, :, None]


def cuda(t):
    return None if t is None else t.cuda()


def kwargs(x, c):
    w = x["w"] or (None, None)
    return dict(positions=cuda(x["pos"]), q_weight=cuda(w[0]), k_weight=cuda(w[1]), eps=EPS,
                interleaved=c[8])


@pytest.mark.parametrize("c", CASES, ids=case_id)
def test_forward(c):
    x = make(c)
    rot, inter, t = c[7], c[8], DTYPES[c[6]]
    q, k, v = split(x["qkv"].cuda(), c)
    got = sdpa_qk_norm_rope(q, k, cuda(x["cos"]), cuda(x["sin"]), v=v, **kwargs(x, c))
    torch.cuda.synchronize()
    cs, sn = turns_of(x, c)
    w = [None if y is None else y.double() for y in (x["w"] or (None, None))]
    for i, (name, part) in enumerate(zip("qk", split(x["qkv"], c))):
        ref, scale = reference(part.double(), w[i], cs, sn, rot, inter)
        check(name, got[i], ref, scale, t)
    assert torch.equal(got[2], v.transpose(1, 2))
    # contiguous inputs and no values: the same bits
    again = sdpa_qk_norm_rope(q.contiguous(), k.contiguous(), cuda(x["cos"]), cuda(x["sin"]),
                              **kwargs(x, c))
    assert again[2] is None and torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("c", CASES, ids=case_id)
def test_backward(c):
    b, s, h, h_kv, d, d_v, dt, rot, inter, wt, _ = c
    x = make(c)
    t = DTYPES[dt]
    g = torch.Generator().manual_seed(5)
    dy = [torch.randn(b, n, s, wd, generator=g).to(t) for n, wd in ((h, d), (h_kv, d), (h_kv, d_v))]
    q, k, v = split(x["qkv"].cuda(), c)
    # the gradients as slices of one fused gradient
    fused = torch.full(x["qkv"].shape, float("nan"), dtype=t, device="cuda")
    dq, dk, dv = split(fused, c)
    kw = kwargs(x, c)
    args = (dy[0].cuda(), dy[1].cuda(), q, k, cuda(x["cos"]), cuda(x["sin"]))
    got = sdpa_qk_norm_rope_bwd(*args, dv_out=dy[2].cuda(), dq=dq, dk=dk, dv=dv, **kw)
    torch.cuda.synchronize()
    assert got[0] is dq and torch.isfinite(fused).all()
    assert torch.equal(dv, dy[2].cuda().transpose(1, 2))
    cs, sn = turns_of(x, c)
    rows_a_thread = b * s * max(h, h_kv)  # more than any thread sums
    for i, part in enumerate(split(x["qkv"], c)[:2]):
        part, w = part.double(), None if wt is None else x["w"][i].double()
        leaves = [part.clone().requires_grad_()] + ([w.clone().requires_grad_()] if wt else [])
        y, _ = reference(leaves[0], leaves[1] if wt else None, cs, sn, rot, inter)
        ref = torch.autograd.grad(y, leaves, dy[i].double())
        gy, gm = turn(dy[i].double().transpose(1, 2), cs, -sn, rot, inter)
        if not wt:
            check("dx", got[i], ref[0], gm, t)
            assert got[3 + i] is None
            continue
        r = (part.square().mean(-1, keepdim=True) + EPS).rsqrt()
        xh = (part * r).abs()
        gw = gm * w.abs()
        check("dx", got[i], ref[0], r * (gw + xh * (gw * xh).mean(-1, keepdim=True)), t)
        chain = min(rows_a_thread, 4 * (rows_a_thread // 600 + 8))
        terms = (gm * xh).sum((0, 1, 2))
        u = torch.finfo(x["w"][i].dtype).eps / 2
        err = (got[3 + i].double().cpu() - ref[1]).abs()
        assert (err <= u * ref[1].abs() + (chain + 80) * 2.0 ** -24 * terms).all()
        assert got[3 + i].dtype == x["w"][i].dtype
    again = sdpa_qk_norm_rope_bwd(*args, **kw)
    assert again[2] is None
    assert torch.equal(again[0], dq) and torch.equal(again[1], dk)


def test_weight_gradients_are_reproducible():
    c = (2, 2048, 8, 2, 128, 128, "bf16", 128, False, "fp32", True)
    x = make(c)
    q, k, _ = split(x["qkv"].cuda(), c)
    dy = [torch.randn(2, n, 2048, 128, device="cuda", dtype=torch.bfloat16) for n in (8, 2)]
    runs = [sdpa_qk_norm_rope_bwd(*dy, q, k, cuda(x["cos"]), cuda(x["sin"]), **kwargs(x, c))
            for _ in range(3)]
    for a in runs[1:]:
        assert all(torch.equal(p, r) for p, r in zip(a, runs[0]) if p is not None)


@pytest.mark.parametrize("d,d_v", [(64, 64), (128, 128), (192, 128)])
def test_cache_rows(d, d_v):
    """Tokens go to rows kv_rows[i] + t of their sequence's cache; tokens that
    fall outside are dropped, every other row stays as it was."""
    b, s, h, h_kv, cap = 5, 6, 4, 2, 20
    c = (b, s, h, h_kv, d, d_v, "bf16", 32, False, "fp32", True)
    x = make(c)
    q, k, v = split(x["qkv"].cuda(), c)
    rows = torch.tensor([0, 14, 17, -3, 20], dtype=torch.int32, device="cuda")
    kw = kwargs(x, c)
    ref = sdpa_qk_norm_rope(q, k, x["cos"].cuda(), x["sin"].cuda(), v=v, **kw)
    # one row of padding behind each head's plane: strides that are not the sizes' products
    kc = torch.randn(b, h_kv, cap + 1, d, device="cuda").bfloat16()
    vc = torch.randn(b, h_kv, cap + 1, d_v, device="cuda").bfloat16()
    want_k, want_v = kc.clone(), vc.clone()
    for i, r in enumerate(rows.tolist()):
        for j in range(s):
            if 0 <= r + j < cap:
                want_k[i, :, r + j] = ref[1][i, :, j]
                want_v[i, :, r + j] = ref[2][i, :, j]
    got = sdpa_qk_norm_rope(q, k, x["cos"].cuda(), x["sin"].cuda(), v=v, kv_rows=rows,
                            k_out=kc[:, :, :cap], v_out=vc[:, :, :cap], **kw)
    torch.cuda.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(kc, want_k) and torch.equal(vc, want_v)


def test_positions_are_held_inside_the_table():
    b, s, h, d = 1, 4, 2, 64
    q = torch.randn(b, s, h, d, device="cuda").half()
    cos, sin = (t.cuda() for t in angles(10, 64))
    pos = torch.tensor([[-7, 0, 9, 1 << 30]], dtype=torch.int32, device="cuda")
    held = torch.tensor([[0, 0, 9, 9]], dtype=torch.int32, device="cuda")
    a = sdpa_qk_norm_rope(q, q, cos, sin, positions=pos)
    r = sdpa_qk_norm_rope(q, q, cos, sin, positions=held)
    assert torch.equal(a[0], r[0]) and torch.equal(a[1], r[1])


def test_zero_rows_and_no_tokens():
    """A row of zeros stays zero and gives no weight gradient; no tokens: empty
    outputs, zero weight gradients."""
    w = torch.ones(64, device="cuda")
    cos, sin = (t.cuda() for t in angles(8, 64))
    for s, eps in ((4, 1e-6), (4, 1e-36), (0, 1e-6)):
        x = torch.zeros(2, s, 3, 64, device="cuda").half()
        q, k, _ = sdpa_qk_norm_rope(x, x, cos, sin, q_weight=w, k_weight=w, eps=eps)
        assert q.shape == (2, 3, s, 64) and not q.any() and not k.any()
        dy = torch.ones(2, 3, s, 64, device="cuda").half()
        g = sdpa_qk_norm_rope_bwd(dy, dy, x, x, cos, sin, q_weight=w, k_weight=w,
                                  dq_weight=torch.full_like(w, 7.0), eps=eps)
        assert not g[3].any() and not g[4].any()
        # dx = g w / sqrt(eps), which at the small eps is beyond fp16: infinite, not NaN
        assert not torch.isnan(g[0]).any() and torch.isfinite(g[0]).all() == (eps > 1e-30)


def test_gradients_against_differences():
    """<grad, dir> against central differences of the fp64 forward."""
    c = (1, 3, 2, 2, 64, 64, "fp16", 32, True, "fp32", True)
    x = make(c)
    g = torch.Generator().manual_seed(2)
    dy = torch.randn(1, 2, 3, 64, generator=g).half()
    q, k, _ = split(x["qkv"].cuda(), c)
    kw = kwargs(x, c)
    got = sdpa_qk_norm_rope_bwd(dy.cuda(), dy.cuda(), q, k, cuda(x["cos"]), cuda(x["sin"]), **kw)
    cs, sn = turns_of(x, c)
    part, w = split(x["qkv"], c)[0].double(), x["w"][0].double()

    def loss(p, wt):
        return (reference(p, wt, cs, sn, 32, True)[0] * dy.double()).sum()

    h = 1e-5
    d = torch.randn(part.shape, generator=g, dtype=torch.float64)
    diff = (loss(part + h * d, w) - loss(part - h * d, w)) / (2 * h)
    # dx is rounded to fp16: off by 2^-11 of itself (2^-25 where tiny)
    dx = got[0].double().cpu()
    assert abs((dx * d).sum() - diff) <= ((2.0 ** -11 * dx.abs() + 2.0 ** -25) * d.abs()).sum() + 1e-6
    e = torch.randn(64, generator=g, dtype=torch.float64)
    diff = (loss(part, w + h * e) - loss(part, w - h * e)) / (2 * h)
    assert abs((got[3].double().cpu() * e).sum() - diff) <= 1e-4


def test_captured_and_on_another_stream():
    c = (2, 40, 4, 2, 128, 128, "bf16", 128, False, "fp32", True)
    x, y = make(c), make((2, 40, 4, 2, 128, 128, "bf16", 128, True, "fp32", True))
    qkv = x["qkv"].cuda()
    q, k, v = split(qkv, c)
    cos, sin = cuda(x["cos"]), cuda(x["sin"])
    kw = kwargs(x, c)

    def step():
        o = sdpa_qk_norm_rope(q, k, cos, sin, v=v, **kw)
        return (*o, *sdpa_qk_norm_rope_bwd(o[0], o[1], q, k, cos, sin, dv_out=o[2], **kw))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    qkv.copy_(y["qkv"] * 0.5)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, eager))


def test_feeds_the_capped_attention():
    """A layer as it is used: fused projection -> norm and rotation -> capped
    attention, and back to one fused gradient; against autograd in fp64 within
    the chained roundings: the attention's inputs are off by u, which moves a
    score by at most 2 u sum|q k| and its output and gradients in proportion;
    checked in the 2-norm at 8 u (u = 2^-8)."""
    b, s, h, h_kv, d, cap = 2, 130, 4, 2, 64, 20.0
    c = (b, s, h, h_kv, d, d, "bf16", 64, False, "fp32", True)
    x = make(c)
    q, k, v = split(x["qkv"].cuda(), c)
    kw = kwargs(x, c)
    cos, sin = cuda(x["cos"]), cuda(x["sin"])
    qa, ka, va = sdpa_qk_norm_rope(q, k, cos, sin, v=v, **kw)
    o, lse = sdpa_fwd(qa, ka, va, is_causal=True, softcap=cap)
    do = torch.randn(o.shape, device="cuda").bfloat16()
    g = sdpa_bwd(qa, ka, va, o, do, lse, is_causal=True, softcap=cap)
    fused = torch.empty_like(x["qkv"], device="cuda")
    dq, dk, dv = split(fused, c)
    r = sdpa_qk_norm_rope_bwd(g[0], g[1], q, k, cos, sin, dv_out=g[2], dq=dq, dk=dk, dv=dv, **kw)
    torch.cuda.synchronize()
    assert sdpa_device_error() == 0
    leaf = x["qkv"].double().requires_grad_()
    w = [t.double().requires_grad_() for t in x["w"]]
    cs, sn = turns_of(x, c)
    parts = split(leaf, c)
    qr = reference(parts[0], w[0], cs, sn, 64, False)[0]
    kr = reference(parts[1], w[1], cs, sn, 64, False)[0].repeat_interleave(h // h_kv, 1)
    vr = parts[2].transpose(1, 2).repeat_interleave(h // h_kv, 1)
    sc = cap * torch.tanh(qr @ kr.transpose(2, 3) / np.sqrt(d) / cap)
    sc = sc.masked_fill(torch.ones(s, s).triu(1).bool(), float("-inf"))
    ref = torch.softmax(sc, -1) @ vr
    grads = torch.autograd.grad(ref, [leaf, *w], do.double().cpu())
    for name, a, e in (("o", o, ref), ("dqkv", fused, grads[0]), ("dqw", r[3], grads[1]),
                       ("dkw", r[4], grads[2])):
        rel = (a.double().cpu() - e).norm() / e.norm()
        assert rel <= 8 * 2.0 ** -8, (name, float(rel))


def test_workspace_too_small():
    x = torch.zeros(1, 8, 2, 64, device="cuda").half()
    dy = torch.zeros(1, 2, 8, 64, device="cuda").half()
    w = torch.ones(64, device="cuda")
    need = sdpa_qk_norm_rope_bwd_workspace_size(1, 8, 2, 2, 64, 64)
    assert need > 0
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        sdpa_qk_norm_rope_bwd(dy, dy, x, x, None, None, q_weight=w, k_weight=w,
                              workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    sdpa_qk_norm_rope_bwd(dy, dy, x, x, None, None, q_weight=w, k_weight=w,
                          workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
