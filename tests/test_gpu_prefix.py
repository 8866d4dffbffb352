"""Attention over a shared prefix and each sequence's own keys
(sdpa_fwd_prefix) against plain fp64 arithmetic, element by element.

Bounds as in capped_bounds (P and O rounded once each, the score's error,
fp32 sums); joining partial rows multiplies each by a weight known to 2^-20
and adds them in fp32, which the 2^-16 of the sums of absolute values covers.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from capped_bounds import u_of
from scaled_dot_product_06_gb300 import (sdpa_device_error, sdpa_fwd, sdpa_fwd_prefix,
                                         sdpa_fwd_prefix_workspace_size, sdpa_qk_norm_rope)
from scaled_dot_product_06_gb300.inputs import DTYPES

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def make(b, h, h_kv, s_q, s_p, s_max, d, d_v, dt, lens, seed=0, q_mul=3.0):
    g = torch.Generator().manual_seed(seed)
    t = DTYPES[dt]

    def r(*shape, mul=1.0):
        return (torch.randn(*shape, generator=g) * mul).to(t)

    x = {"q": r(b, h, s_q, d, mul=q_mul), "kp": r(h_kv, s_p, d), "vp": r(h_kv, s_p, d_v),
         "k": r(b, h_kv, s_max, d), "v": r(b, h_kv, s_max, d_v)}
    for i, n in enumerate(lens):  # behind the last key: anything
        n = min(max(n, 0), s_max)
        x["k"][i, :, n:] = float("nan")
        x["v"][i, :, n:] = float("inf") if i % 2 else float("nan")
    x["lens"] = torch.tensor(lens, dtype=torch.int32)
    return x


def call(x, **kw):
    return sdpa_fwd_prefix(*(x[n].cuda() for n in ("q", "kp", "vp", "k", "v", "lens")), **kw)


def reference(x, scale, cap):
    """(o, lse) and their bounds."""
    b, h, s_q, d = x["q"].shape
    h_kv, s_p = x["kp"].shape[:2]
    s_max, d_v = x["v"].shape[2:]
    u = u_of(x["q"].dtype)
    sub = 2.0 ** -25 if x["q"].dtype == torch.float16 else 0.0
    o, oe = np.zeros((b, h, s_q, d_v)), np.zeros((b, h, s_q, d_v))
    lse, le = np.zeros((b, h, s_q)), np.zeros((b, h, s_q))
    for i in range(b):
        n = min(max(int(x["lens"][i]), 0), s_max)
        for j in range(h):
            hk = j // (h // h_kv)
            k = np.concatenate((f64(x["kp"][hk]), f64(x["k"][i, hk, :n])))
            v = np.concatenate((f64(x["vp"][hk]), f64(x["v"][i, hk, :n])))
            q = f64(x["q"][i, j])
            s = scale * (q @ k.T)
            e_s = abs(scale) * (np.abs(q) @ np.abs(k).T) * d * 2.0 ** -24
            if cap:
                s = cap * np.tanh(s / cap)
                e_s = e_s + cap * 2.0 ** -20
            own = np.arange(s_p + n)[None] - s_p  # negative: the prefix, seen by all
            seen = (own < 0) | (own <= (n - s_q + np.arange(s_q))[:, None])
            for t in range(s_q):
                vis = seen[t]
                if not vis.any():
                    lse[i, j, t] = -np.inf
                    continue
                m = s[t, vis].max()
                p = np.where(vis, np.exp(np.where(vis, s[t], m) - m), 0.0)
                lse[i, j, t] = m + np.log(p.sum())
                p = p / p.sum()
                es = e_s[t, vis].max()
                o[i, j, t] = p @ v
                oe[i, j, t] = ((u + 2 * es + 2.0 ** -20 + 2.0 ** -16) * p + 256 * sub * vis) @ np.abs(v) \
                    + u * np.abs(o[i, j, t]) + sub
                le[i, j, t] = es + 2.0 ** -19 * (1 + abs(lse[i, j, t]) + cap)
    return o, lse, oe, le


def check(x, got, scale, cap):
    torch.cuda.synchronize()
    assert sdpa_device_error() == 0
    o, lse, oe, le = reference(x, scale, cap)
    for name, a, r, e in (("o", got[0], o, oe), ("lse", got[1], lse, le)):
        a = f64(a)
        ninf = np.isneginf(r)
        assert np.array_equal(np.isneginf(a), ninf), name
        assert np.isfinite(a[~ninf]).all(), name
        over = np.abs(a[~ninf] - r[~ninf]) - e[~ninf]
        assert over.size == 0 or over.max() <= 0, (
            f"{name}: {int((over > 0).sum())} of {over.size} past their bound by {over.max():.3e}")


# (b, h, h_kv, s_q, s_prefix, s_max, lens, d, d_v, dtype, cap)
CASES = [
    (3, 8, 2, 1, 300, 200, [1, 130, 200], 128, 128, "bf16", 0.0),
    (2, 8, 1, 1, 333, 17, [1, 17], 64, 64, "bf16", 0.0),
    (2, 4, 4, 4, 513, 260, [4, 259], 192, 128, "fp16", 30.0),
    (1, 1, 1, 1, 1, 1, [1], 64, 64, "fp16", 0.0),
    (3, 4, 2, 2, 0, 300, [2, 129, 256], 128, 128, "bf16", 20.0),       # no prefix
    (4, 4, 2, 3, 257, 0, [0, 0, 0, 0], 128, 128, "bf16", 0.0),         # no own keys
    (2, 2, 1, 3, 0, 64, [0, 2], 64, 64, "fp16", 0.0),                  # rows that see nothing
    (2, 4, 1, 2, 128, 128, [0, 128], 64, 64, "bf16", 10.0),            # none, all, whole tiles
    (40, 12, 4, 1, 700, 90, list(range(1, 81, 2)), 128, 128, "bf16", 0.0),   # 42 sequences a row tile
    (19, 16, 1, 1, 1300, 64, [64 - i for i in range(19)], 64, 64, "fp16", 0.0),  # odd row tiles
    (2, 16, 1, 9, 400, 500, [9, 444], 128, 128, "bf16", 0.0),          # R = 144: two tiles of own rows
    (2, 32, 1, 10, 260, 300, [300, 10], 64, 64, "bf16", 15.0),         # R = 320: three
    (1, 8, 1, 16, 3000, 1000, [1000], 128, 128, "fp16", 0.0),          # R = 128
    (1, 8, 8, 1, 40000, 20, [20], 64, 64, "bf16", 0.0),                # a long prefix, many parts
    (5, 10, 2, 1, 0, 9000, [9000, 1, 4097, 8999, 128], 128, 128, "bf16", 0.0),  # long own keys
    (2, 4, 2, 1, 130, 50, [77, -3], 64, 64, "bf16", 0.0),              # lengths outside the cache
    (2, 4, 2, 5, 5000, 4000, [4000, 3], 192, 128, "bf16", 0.0),        # fewer keys than tokens
    (2, 16, 1, 9, 400, 500, [9, 444], 192, 128, "bf16", 0.0),          # row tiles one by one: R = 144
    (40, 12, 4, 1, 700, 90, list(range(1, 81, 2)), 192, 128, "fp16", 20.0),  # and of the prefix
    (2, 32, 1, 1, 0, 1100, [1100, 33], 128, 128, "bf16", 0.0),         # R = 32: all lanes of a warp
    (2, 33, 1, 1, 60, 300, [300, 97], 64, 64, "fp16", 30.0),           # R = 33: one more
    (200, 8, 1, 1, 0, 900, [900 if i % 37 == 5 else i % 2 for i in range(200)], 64, 64, "bf16", 0.0),  # more
    # items than CTAs, most of them empty
    (200, 4, 1, 1, 0, 40, [0] * 200, 64, 64, "bf16", 10.0),            # all of them
]


def case_id(c):
    return f"b{c[0]}h{c[1]}kv{c[2]}q{c[3]}-p{c[4]}-own{c[5]}-d{c[7]}x{c[8]}-{c[9]}-cap{c[10]}"


@pytest.mark.parametrize("c", CASES, ids=case_id)
def test_matches_reference(c):
    b, h, h_kv, s_q, s_p, s_max, lens, d, d_v, dt, cap = c
    x = make(b, h, h_kv, s_q, s_p, s_max, d, d_v, dt, lens, seed=len(lens) + s_p)
    got = call(x, softcap=cap)
    check(x, got, 1.0 / np.sqrt(d), cap)
    again = call(x, softcap=cap)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("scale", [-0.2, 0.0])
@pytest.mark.parametrize("cap", [0.0, 7.0])
def test_negative_and_zero_scale(scale, cap):
    x = make(2, 4, 2, 2, 200, 140, 64, 64, "bf16", [139, 2])
    check(x, call(x, scale=scale, softcap=cap), scale, cap)


def test_scores_at_the_cap_and_far_apart():
    """Scores that saturate the cap, and a running maximum that jumps between
    key tiles and partials."""
    x = make(2, 8, 2, 1, 900, 300, 128, 128, "bf16", [300, 45], q_mul=40.0)
    x["kp"][:, 500] *= 8
    check(x, call(x, softcap=20.0), 1 / np.sqrt(128), 20.0)
    y = make(2, 8, 2, 1, 900, 300, 128, 128, "bf16", [300, 45], q_mul=6.0)
    y["kp"][:, 500] *= 8
    y["k"][0, :, 200] *= 12
    check(y, call(y), 1 / np.sqrt(128), 0.0)


def test_writes_stay_inside():
    """Outputs and workspace in the middle of larger buffers, whose other bytes
    keep their values; the inputs keep theirs."""
    x = make(3, 6, 2, 2, 300, 150, 128, 128, "bf16", [2, 150, 77])
    need = sdpa_fwd_prefix_workspace_size(3, 6, 2, 2, 300, 150, 128, 128)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    buf = torch.full((3 * 6 * 2 * 128 + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    lb = torch.full((3 * 6 * 2 + 8,), 7.0, device="cuda")
    gpu = {n: t.cuda() for n, t in x.items()}
    before = {n: t.clone() for n, t in gpu.items()}
    out, lse = buf[64:-64].view(3, 6, 2, 128), lb[4:-4].view(3, 6, 2)
    got = sdpa_fwd_prefix(gpu["q"], gpu["kp"], gpu["vp"], gpu["k"], gpu["v"], gpu["lens"], out=out, lse=lse,
                          workspace=ws[256:256 + need])
    assert got[0] is out
    check(x, got, 1 / np.sqrt(128), 0.0)
    assert (ws[:256] == 0x5A).all() and (ws[256 + need:] == 0x5A).all()
    assert (buf[:64] == 7).all() and (buf[-64:] == 7).all() and (lb[:4] == 7).all() and (lb[-4:] == 7).all()
    for n, t in gpu.items():
        assert torch.equal(t.view(torch.int16) if t.dtype == torch.bfloat16 else t,
                           before[n].view(torch.int16) if t.dtype == torch.bfloat16 else before[n]), n


@pytest.mark.parametrize("d,d_v", [(64, 64), (128, 128), (192, 128)])
def test_what_lies_behind_the_last_key_under_load(d, d_v):
    """Every SM streaming, ragged lengths: the results with NaN behind the last
    keys are, bit for bit, those with zeros there."""
    b, h, h_kv, s_p, s_max = 64, 16, 4, 2000, 900
    g = torch.Generator().manual_seed(8)
    lens = torch.randint(1, s_max + 1, (b,), generator=g).tolist()
    x = make(b, h, h_kv, 1, s_p, s_max, d, d_v, "bf16", lens)
    y = dict(x, k=torch.nan_to_num(x["k"], 0.0), v=torch.nan_to_num(x["v"], 0.0, 0.0, 0.0))
    gx, gy = ([t[n].cuda() for n in ("q", "kp", "vp", "k", "v", "lens")] for t in (x, y))
    want = sdpa_fwd_prefix(*gy)
    assert torch.isfinite(want[0]).all()
    for _ in range(10):
        got = sdpa_fwd_prefix(*gx)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert sdpa_device_error() == 0


def test_two_streams_and_a_graph():
    """Two calls at once with a workspace each, and a captured call replayed
    after the cache has grown, give the bits of the calls one by one."""
    a = make(4, 8, 2, 1, 2000, 600, 128, 128, "bf16", [1, 600, 333, 128], seed=1)
    b = make(4, 8, 2, 1, 1500, 600, 128, 128, "bf16", [600, 2, 77, 555], seed=2)
    ga, gb = ({n: t.cuda() for n, t in x.items()} for x in (a, b))

    def run(g, **kw):
        return sdpa_fwd_prefix(g["q"], g["kp"], g["vp"], g["k"], g["v"], g["lens"], softcap=30.0, **kw)

    alone = [run(ga), run(gb)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        r1 = run(ga, stream=s1)
        r2 = run(gb, stream=s2)
        torch.cuda.synchronize()
        for r, e in ((r1, alone[0]), (r2, alone[1])):
            assert torch.equal(r[0], e[0]) and torch.equal(r[1], e[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(ga)
    for n in ("q", "k", "v", "lens"):
        ga[n].copy_(b[n])
    graph.replay()
    torch.cuda.synchronize()
    e = run(ga)
    assert torch.equal(out[0], e[0]) and torch.equal(out[1], e[1])
    assert sdpa_device_error() == 0


def test_graphs_share_a_workspace():
    """More items than CTAs (the counter is cleared in the graph): two graphs with
    one workspace, replayed in turn with other lengths, give the eager calls' bits."""
    calls, want = [], []
    b, h, h_kv, s_max, d = 180, 4, 1, 500, 64
    size = sdpa_fwd_prefix_workspace_size(b, h, h_kv, 1, 300, s_max, d, d)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)
    for seed in (1, 2):
        x = make(b, h, h_kv, 1, 300, s_max, d, d, "bf16", [s_max] * b, seed=seed)
        args = [x[n].cuda() for n in ("q", "kp", "vp", "k", "v", "lens")]
        out = (torch.empty(b, h, 1, d, dtype=torch.bfloat16, device="cuda"),
               torch.empty(b, h, 1, device="cuda"))
        kw = dict(out=out[0], lse=out[1], workspace=ws)
        sdpa_fwd_prefix(*args, **kw)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sdpa_fwd_prefix(*args, **kw)
        calls.append((graph, args, out))
    for turn in range(3):
        for graph, args, out in calls:
            args[5].copy_(torch.tensor([(37 * i + 101 * turn) % (s_max + 1) for i in range(b)]))
            want.append([t.clone() for t in sdpa_fwd_prefix(*args)])
            out[0].zero_(), out[1].zero_()
            graph.replay()
            assert torch.equal(out[0], want[-1][0]) and torch.equal(out[1], want[-1][1])
    torch.cuda.synchronize()
    assert sdpa_device_error() == 0


def test_serving_loop_equals_the_whole_sequence():
    """As it is served: the prompt's keys normed, rotated and attended once,
    then tokens normed, rotated, appended and attended one step at a time; each
    step equals the capped attention over the whole sequence of that moment.
    Both sides round P and O once (u each) from the same bf16 keys: within
    4 u of sum P |V|, at most 4 u max|V|."""
    b, h, h_kv, d, s_p, cap_rows, steps, cap = 3, 8, 2, 128, 200, 40, 4, 25.0
    g = torch.Generator().manual_seed(4)
    t = torch.bfloat16
    pos = torch.arange(1000, dtype=torch.float64)[:, None]
    ang = pos * 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    cos, sin = ang.cos().float().cuda(), ang.sin().float().cuda()
    w = [(1 + 0.1 * torch.randn(d, generator=g)).cuda() for _ in range(2)]
    kw = dict(q_weight=w[0], k_weight=w[1])

    def project(n, s):
        y = torch.randn(n, s, (h + 2 * h_kv) * d, generator=g).to(t).cuda()
        return (y[..., :h * d].unflatten(-1, (h, d)), y[..., h * d:(h + h_kv) * d].unflatten(-1, (h_kv, d)),
                y[..., (h + h_kv) * d:].unflatten(-1, (h_kv, d)))

    q, k, v = project(1, s_p)
    _, kp, vp = sdpa_qk_norm_rope(q, k, cos, sin, v=v, **kw)
    kc = torch.full((b, h_kv, cap_rows, d), float("nan"), dtype=t, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    lens = torch.tensor([0, 7, 30], dtype=torch.int32, device="cuda")
    for i, n in enumerate(lens.tolist()):  # what the sequences have said so far
        kc[i, :, :n] = torch.randn(h_kv, n, d, generator=g).to(t).cuda()
        vc[i, :, :n] = torch.randn(h_kv, n, d, generator=g).to(t).cuda()
    for step in range(steps):
        s = 1 + step % 2
        q, k, v = project(b, s)
        positions = (s_p + lens[:, None] + torch.arange(s, device="cuda")).to(torch.int32)
        qn, _, _ = sdpa_qk_norm_rope(q, k, cos, sin, v=v, positions=positions, kv_rows=lens, k_out=kc,
                                     v_out=vc, **kw)
        lens += s
        o, lse = sdpa_fwd_prefix(qn, kp[0], vp[0], kc, vc, lens, softcap=cap)
        for i, n in enumerate(lens.tolist()):
            kk = torch.cat((kp, kc[i:i + 1, :, :n]), 2).contiguous()
            vv = torch.cat((vp, vc[i:i + 1, :, :n]), 2).contiguous()
            ow, lw = sdpa_fwd(qn[i:i + 1].contiguous(), kk, vv, is_causal=True, bottom_right=True, softcap=cap)
            assert (o[i:i + 1] - ow).abs().max() <= 4 * 2.0 ** -8 * vv.abs().max()
            assert (lse[i:i + 1] - lw).abs().max() <= 1e-4
    torch.cuda.synchronize()
    assert sdpa_device_error() == 0


def test_refusals():
    x = {n: t.cuda() for n, t in make(2, 4, 2, 1, 16, 16, 64, 64, "bf16", [1, 1]).items()}
    args = [x[n] for n in ("q", "kp", "vp", "k", "v", "lens")]
    for i, bad in ((1, x["kp"][:1]), (2, x["vp"].half()), (3, x["k"].transpose(2, 3)), (5, x["lens"].long()),
                   (5, x["lens"][:1]), (5, x["lens"].cpu())):
        a = list(args)
        a[i] = bad
        with pytest.raises(ValueError):
            sdpa_fwd_prefix(*a)
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        sdpa_fwd_prefix(*args, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(RuntimeError, match="softcap"):
        sdpa_fwd_prefix(*args, softcap=-2.0)
    with pytest.raises(RuntimeError, match="scale"):
        sdpa_fwd_prefix(*args, scale=float("inf"))
