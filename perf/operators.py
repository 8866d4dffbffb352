"""What is measured of the operators around the attention call: the norm and
rotation of queries and keys, attention with capped scores, and attention of
new tokens over a prefix that their batch shares.

``run`` computes a case in plain torch operations (fp32, rounded once at the
end) or, where ``own`` is true, through the package's entry points. ``exact``
computes the same in 64 bits, one batch entry and head at a time, with
gradients from autograd.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- the cases
def _norm(name, way, b, s, h, h_kv, d, d_v, dtype, rot, interleaved=False, rows=0, normed=True):
    """way: fwd (BHSD outputs), append (K and V rows of a cache of `rows`), bwd."""
    return {"name": name, "op": "norm", "way": way, "b": b, "s": s, "h": h, "h_kv": h_kv, "d": d,
            "d_v": d_v, "dtype": dtype, "rot": rot, "interleaved": interleaved, "rows": rows,
            "normed": normed}


def _cap(name, way, b, h, h_kv, s_q, s_kv, d, d_v, dtype, cap, left=-1, right=-1, lens=0,
         bottom_right=False):
    """way: fwd, step (forward and backward); lens != 0: b packed sequences of
    at most s_q = s_kv tokens, their lengths drawn from it."""
    return {"name": name, "op": "cap", "way": way, "b": b, "h": h, "h_kv": h_kv, "s_q": s_q,
            "s_kv": s_kv, "d": d, "d_v": d_v, "dtype": dtype, "cap": cap, "left": left,
            "right": right, "lens": lens, "bottom_right": bottom_right}


def _prefix(name, b, h, h_kv, s_q, d, d_v, dtype, prefix, rows, lens, cap=0.0):
    """b sequences of s_q new tokens, `prefix` shared keys, caches of `rows`."""
    return {"name": name, "op": "prefix", "b": b, "h": h, "h_kv": h_kv, "s_q": s_q, "d": d,
            "d_v": d_v, "dtype": dtype, "prefix": prefix, "rows": rows, "lens": lens, "cap": cap}


def listed():
    return [
        # one decoding step of a served batch: norm, rotate and append one token of each sequence
        _norm("norm-append-b64", "append", 64, 1, 32, 4, 128, 128, "bf16", 128, rows=1024),
        # a long prompt or a training sequence with grouped heads
        _norm("norm-fwd-s16384", "fwd", 1, 16384, 32, 4, 128, 128, "bf16", 128),
        # odd prompt lengths into caches, adjacent pairs rotated, part of a wide head
        _norm("norm-append-odd-d192", "append", 3, 777, 12, 3, 192, 128, "fp16", 64, True, rows=1000),
        # the backward pass of a training batch
        _norm("norm-bwd-b4-s2048", "bwd", 4, 2048, 16, 16, 128, 128, "bf16", 128),
        # the smallest attention call, where latency counts
        _cap("cap-fwd-b1h2-s128", "fwd", 1, 2, 2, 128, 128, 64, 64, "bf16", 30.0, right=0),
        # cross lengths without a mask, small heads
        _cap("cap-fwd-s1024x2048-d64", "fwd", 8, 16, 16, 1024, 2048, 64, 64, "fp16", 30.0),
        # a training step of a batch
        _cap("cap-step-b4h16-s2048", "step", 4, 16, 16, 2048, 2048, 128, 128, "bf16", 50.0, right=0),
        # a training step with a sliding window over a long sequence, grouped heads
        _cap("cap-step-window4096", "step", 1, 32, 4, 8192, 8192, 128, 128, "bf16", 50.0, left=4096,
             right=0),
        # a training step over packed documents of ragged lengths
        _cap("cap-step-packed16", "step", 16, 8, 8, 1500, 1500, 128, 128, "bf16", 50.0, right=0,
             lens=7),
        # two sequences just begun behind a short common prompt
        _prefix("prefix-b2-p333", 2, 8, 1, 1, 64, 64, "bf16", 333, 17, 1),
        # a served batch behind a long common prompt
        _prefix("prefix-b64-p16384", 64, 32, 4, 1, 128, 128, "bf16", 16384, 1024, 2, 50.0),
        # four drafted tokens at a time, one K/V head a query head, wide heads
        _prefix("prefix-draft4-d192", 16, 16, 16, 4, 192, 128, "fp16", 2048, 600, 3),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_once(rng):
    op = rng.choice(("norm", "cap", "prefix"))
    dtype = rng.choice(("bf16", "fp16"))
    d, d_v = rng.choice(((64, 64), (128, 128), (192, 128)))
    h_kv = rng.choice((1, 2, 3, 4, 8, 16))
    h = h_kv * rng.choice((1, 2, 4, 5, 8))
    if op == "norm":
        way = rng.choice(("fwd", "append", "bwd"))
        s = _log(rng, 1, 8192)
        return _norm(None, way, _log(rng, 1, 64), s, h, h_kv, d, d_v, dtype,
                     rng.choice((16, 32, 48, 64, d)), rng.random() < 0.4,
                     rows=s + rng.randrange(0, 64), normed=rng.random() < 0.8)
    cap = rng.choice((10.0, 20.0, 30.0, 50.0))
    if op == "cap":
        way = rng.choice(("fwd", "step"))
        # the gradient through a softmax over a single key is zero: nothing to measure against
        least = 64 if way == "step" else 1
        s_q = _log(rng, least, 4096)
        left, right = rng.choice(((-1, -1), (-1, 0), (_log(rng, 16, 2048), 0), (100, 50)))
        if rng.random() < 0.3:
            return _cap(None, way, rng.randrange(1, 17), h, h_kv, s_q, s_q, d, d_v, dtype, cap, left,
                        right, lens=rng.randrange(1, 1000))
        s_kv = s_q if rng.random() < 0.5 else _log(rng, least, 4096)
        return _cap(None, way, _log(rng, 1, 16), h, h_kv, s_q, s_kv, d, d_v, dtype, cap, left, right,
                    bottom_right=rng.random() < 0.3)
    s_q = rng.choice((1, 1, 1, 2, 3, 5, 8))
    return _prefix(None, _log(rng, 1, 96), h, h_kv, s_q, d, d_v, dtype,
                   rng.choice((0, _log(rng, 1, 40000), _log(rng, 100, 40000))),
                   s_q + _log(rng, 1, 4000), rng.randrange(1, 1000), rng.choice((0.0, cap)))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        for k in ("bytes", "flops"):
            most[c["op"], k] = max(most.get((c["op"], k), 0), w[k])
    while True:
        c = _draw_once(rng)
        c.pop("name")
        w = work(c)
        # scores the plain form holds at once, as the largest listed case does
        scores = c["b"] * c["h"] * c["s_q"] * c["s_kv"] if c["op"] == "cap" else 0
        if scores <= 32 * 8192 * 8192 and all(w[k] <= most[c["op"], k] for k in w):
            return c


def _lengths(c):
    """Packed lengths: from one token to the longest, one of them the longest."""
    rng = random.Random(c["lens"])
    n = [rng.randrange(1, c["s_q"] + 1) for _ in range(c["b"])]
    n[rng.randrange(c["b"])] = c["s_q"]
    return n


def _own_lengths(c):
    """Tokens of each cache, the new ones among them."""
    rng = random.Random(c["lens"])
    return [rng.randrange(c["s_q"], c["rows"] + 1) for _ in range(c["b"])]


def _pairs(s_q, s_kv, left, right, bottom_right):
    """Visible (query, key) pairs of one head."""
    off = s_kv - s_q if bottom_right else 0
    n = 0
    for i in range(s_q):
        lo = 0 if left < 0 else max(0, i + off - left)
        hi = s_kv - 1 if right < 0 else min(s_kv - 1, i + off + right)
        n += max(0, hi - lo + 1)
    return n


def work(case):
    c = case
    if c["op"] == "norm":
        el = c["b"] * c["s"] * ((c["h"] + c["h_kv"]) * c["d"] + c["h_kv"] * c["d_v"])
        v = c["b"] * c["s"] * c["h_kv"] * c["d_v"]
        table = c["b"] * c["s"] * c["rot"] * 4
        if c["way"] == "bwd":
            return {"bytes": 2 * (3 * (el - v) + 2 * v) + table, "flops": 20 * (el - v)}
        return {"bytes": 2 * 2 * el + table, "flops": 10 * (el - v)}
    if c["op"] == "cap":
        if c["lens"]:
            n = _lengths(c)
            tq = tk = sum(n)
            pairs = sum(_pairs(x, x, c["left"], c["right"], c["bottom_right"]) for x in n)
        else:
            tq, tk = c["b"] * c["s_q"], c["b"] * c["s_kv"]
            pairs = c["b"] * _pairs(c["s_q"], c["s_kv"], c["left"], c["right"], c["bottom_right"])
        d, d_v = c["d"], c["d_v"]
        q, kv, o = tq * c["h"] * d, tk * c["h_kv"] * (d + d_v), tq * c["h"] * d_v
        flops, size = 2 * (d + d_v) * pairs * c["h"], 2 * (q + kv + o) + 4 * tq * c["h"]
        if c["way"] == "step":
            flops += 2 * (3 * d + 2 * d_v) * pairs * c["h"]
            size += 2 * (q + kv + o)
        return {"bytes": size, "flops": flops}
    n = _own_lengths(c)
    d, d_v = c["d"], c["d_v"]
    pairs = sum(c["s_q"] * (c["prefix"] + x) - c["s_q"] * (c["s_q"] - 1) // 2 for x in n) * c["h"]
    rows = c["b"] * c["h"] * c["s_q"]
    return {"bytes": 2 * (d + d_v) * (c["h_kv"] * (c["prefix"] + sum(n)) + rows) + 4 * rows,
            "flops": 2 * (d + d_v) * pairs}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    t = DTYPES[c["dtype"]]

    def randn(*shape, mul=1.0, dtype=t):
        return (torch.randn(*shape, generator=g, device=dev) * mul).to(dtype)

    st = {"case": dict(c)}
    if c["op"] == "norm":
        b, s, h, h_kv, d, d_v, rot = (c[k] for k in ("b", "s", "h", "h_kv", "d", "d_v", "rot"))
        # the fused projection's output, and its parts as views
        qkv = randn(b, s, h * d + h_kv * (d + d_v), mul=2.0)
        st["q"] = qkv[..., :h * d].unflatten(-1, (h, d))
        st["k"] = qkv[..., h * d:(h + h_kv) * d].unflatten(-1, (h_kv, d))
        st["v"] = qkv[..., (h + h_kv) * d:].unflatten(-1, (h_kv, d_v))
        st["q_weight"] = st["k_weight"] = None
        if c["normed"]:
            st["q_weight"] = 1.0 + randn(d, mul=0.1, dtype=torch.float32)
            st["k_weight"] = 1.0 + randn(d, mul=0.1, dtype=torch.float32)
        # each sequence has come to a position of its own
        base = torch.randint(0, 30000, (b, 1), generator=g, device=dev)
        n_pos = 30000 + s
        inv = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=dev),
                        -torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
        ang = torch.arange(n_pos, dtype=torch.float64, device=dev)[:, None] * inv
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        st["positions"] = (base + torch.arange(s, device=dev)).to(torch.int32)
        if c["way"] == "append":
            st["kv_rows"] = torch.randint(0, c["rows"] - s + 1, (b,), generator=g,
                                          device=dev).to(torch.int32)
            st["k_cache"] = randn(b, h_kv, c["rows"], d)
            st["v_cache"] = randn(b, h_kv, c["rows"], d_v)
        if c["way"] == "bwd":
            st["dq_out"], st["dk_out"] = randn(b, h, s, d), randn(b, h_kv, s, d)
            st["dv_out"] = randn(b, h_kv, s, d_v)
        return st
    b, h, h_kv, d, d_v, s_q = (c[k] for k in ("b", "h", "h_kv", "d", "d_v", "s_q"))
    st["scale"] = 1.0 / math.sqrt(d)
    if c["op"] == "cap":
        if c["lens"]:
            n = _lengths(c)
            starts = [0]
            for x in n:
                starts.append(starts[-1] + x)
            st["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
            lead, rows_q, rows_k = (), starts[-1], starts[-1]
        else:
            lead, rows_q, rows_k = (b,), s_q, c["s_kv"]
        # queries large enough that the scores reach the cap's bend
        st["q"], st["k"] = randn(*lead, h, rows_q, d, mul=4.0), randn(*lead, h_kv, rows_k, d)
        st["v"] = randn(*lead, h_kv, rows_k, d_v)
        st["do"] = randn(*lead, h, rows_q, d_v)
        return st
    n = _own_lengths(c)
    st["q"] = randn(b, h, s_q, d, mul=2.0)
    st["k_prefix"], st["v_prefix"] = randn(h_kv, c["prefix"], d), randn(h_kv, c["prefix"], d_v)
    st["k"], st["v"] = randn(b, h_kv, c["rows"], d), randn(b, h_kv, c["rows"], d_v)
    st["lens"] = torch.tensor(n, dtype=torch.int32, device=dev)
    # what lies behind a sequence's last token in its cache is whatever was there before
    behind = torch.arange(c["rows"], device=dev)[None, :] >= st["lens"][:, None]
    st["k"].masked_fill_(behind[:, None, :, None], float("nan"))
    st["v"].masked_fill_(behind[:, None, :, None], float("nan"))
    return st


# ---------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, rot, interleaved):
    """The first `rot` elements of x's last dimension rotated; cos, sin broadcast to x."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


EPS = 1e-6


def _norm_plain(st):
    c = st["case"]
    t, rot, inter = DTYPES[c["dtype"]], c["rot"], c["interleaved"]
    pos = st["positions"].long()
    cos, sin = st["cos"][pos][:, :, None], st["sin"][pos][:, :, None]  # [b, s, 1, rot / 2]

    def forward(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        return _rotate(x, cos, sin, rot, inter).transpose(1, 2).to(t)

    def backward(dy, x, w):
        g = _rotate(dy.float().transpose(1, 2), cos, -sin, rot, inter)
        if w is None:
            return g.to(t).contiguous(), None
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        xh = x * r
        gw = g * w
        dx = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
        return dx.to(t), (g * xh).sum((0, 1, 2))

    if c["way"] == "bwd":
        dq, dqw = backward(st["dq_out"], st["q"], st["q_weight"])
        dk, dkw = backward(st["dk_out"], st["k"], st["k_weight"])
        return dq, dk, st["dv_out"].transpose(1, 2).contiguous(), dqw, dkw
    q, k = forward(st["q"], st["q_weight"]), forward(st["k"], st["k_weight"])
    v = st["v"].transpose(1, 2)
    if c["way"] == "fwd":
        return q.contiguous(), k.contiguous(), v.contiguous()
    bi = torch.arange(c["b"], device=q.device)[:, None, None]
    hi = torch.arange(c["h_kv"], device=q.device)[None, :, None]
    ri = st["kv_rows"].long()[:, None, None] + torch.arange(c["s"], device=q.device)
    st["k_cache"][bi, hi, ri] = k
    st["v_cache"][bi, hi, ri] = v
    return q.contiguous(), st["k_cache"], st["v_cache"]


def _visible(rows, cols, s_q, s_kv, c):
    off = s_kv - s_q if c["bottom_right"] else 0
    d = cols - rows - off
    ok = torch.ones_like(d, dtype=torch.bool)
    if c["left"] >= 0:
        ok &= d >= -c["left"]
    if c["right"] >= 0:
        ok &= d <= c["right"]
    return ok


def _softmax(s, visible):
    """P and the natural logsumexp of masked scores; a row that sees no key: 0, -inf."""
    s = s.masked_fill_(~visible, float("-inf"))
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(s - m0)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    return p, (m0 + torch.log(total)).squeeze(-1)


def _cap_plain(st):
    c = st["case"]
    t, cap, scale = DTYPES[c["dtype"]], c["cap"], st["scale"]
    q, k, v = st["q"], st["k"], st["v"]
    dev = q.device
    if c["lens"]:
        # padded to the longest: rows[i] are sequence i's tokens, past its end its last one again
        n = (st["starts"][1:] - st["starts"][:-1]).long()
        at = torch.arange(c["s_q"], device=dev)
        rows = st["starts"][:-1].long()[:, None] + torch.minimum(at, n[:, None] - 1)  # [b, s]
        live = at < n[:, None]
        q, k, v, do = (x[:, rows].transpose(0, 1) for x in (q, k, v, st["do"]))
        visible = (_visible(at[:, None], at[None, :], c["s_q"], c["s_kv"], c)[None]
                   & live[:, None, :] & live[:, :, None])[:, None, None]
        do = do * live[:, None, :, None]
    else:
        visible = _visible(torch.arange(c["s_q"], device=dev)[:, None],
                           torch.arange(c["s_kv"], device=dev)[None, :], c["s_q"], c["s_kv"], c)
        do = st["do"]
    b, s_q, grp = q.shape[0], q.shape[2], c["h"] // c["h_kv"]
    q = q.float().unflatten(1, (c["h_kv"], grp))  # [b, h_kv, group, s_q, d]
    k, v = k.float()[:, :, None], v.float()[:, :, None]
    tanh = torch.tanh(torch.matmul(q, k.mT) * (scale / cap))
    p, lse = _softmax(tanh * cap, visible)
    o = torch.matmul(p, v)

    def rows_of(x):  # [b, heads, s, ...] to the packed rows
        if not c["lens"]:
            return x
        return x.transpose(0, 1).flatten(1, 2)[:, live.flatten()]

    out = [rows_of(o.flatten(1, 2).to(t)), rows_of(lse.flatten(1, 2))]
    if c["way"] == "step":
        do = do.float().unflatten(1, (c["h_kv"], grp))
        dv = torch.matmul(p.mT, do).sum(2)
        ds = torch.matmul(do, v.mT)
        ds -= (do * o).sum(-1, keepdim=True)
        ds *= p
        ds *= 1.0 - tanh.square()
        dq = torch.matmul(ds, k) * scale
        dk = torch.matmul(ds.mT, q).sum(2) * scale
        out += [rows_of(dq.flatten(1, 2).to(t)), rows_of(dk.to(t)), rows_of(dv.to(t))]
    return tuple(x.contiguous() for x in out)


def _prefix_plain(st):
    c = st["case"]
    t, s_q, grp = DTYPES[c["dtype"]], c["s_q"], c["h"] // c["h_kv"]
    q = st["q"].float().unflatten(1, (c["h_kv"], grp)).flatten(2, 3)  # [b, h_kv, group * s_q, d]
    at = torch.arange(c["rows"], device=q.device)
    behind = (at >= st["lens"][:, None])[:, None, :, None]
    k = st["k"].float().masked_fill_(behind, 0.0)
    v = st["v"].float().masked_fill_(behind, 0.0)
    kp, vp = st["k_prefix"].float(), st["v_prefix"].float()
    s = torch.cat((torch.matmul(q, kp.mT), torch.matmul(q, k.mT)), -1) * st["scale"]
    if c["cap"] > 0:
        s = torch.tanh(s / c["cap"]) * c["cap"]
    # new token i of a sequence sees its own keys up to its own place
    last = st["lens"][:, None] - s_q + torch.arange(s_q, device=q.device)  # [b, s_q]
    seen = at <= last[:, :, None]
    seen = torch.cat((seen.new_ones(c["b"], s_q, c["prefix"]), seen), -1)
    p, lse = _softmax(s, seen[:, None].repeat(1, 1, grp, 1))
    o = torch.matmul(p[..., :c["prefix"]], vp) + torch.matmul(p[..., c["prefix"]:], v)
    o = o.unflatten(2, (grp, s_q)).flatten(1, 2).to(t)
    return o, lse.unflatten(2, (grp, s_q)).flatten(1, 2)


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _norm_own, "cap": _cap_own, "prefix": _prefix_own}[op](state)
    return {"norm": _norm_plain, "cap": _cap_plain, "prefix": _prefix_plain}[op](state)


def _norm_own(st):
    import scaled_dot_product_06_gb300 as sdpa
    c = st["case"]
    kw = dict(positions=st["positions"], q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS,
              interleaved=c["interleaved"])
    if c["way"] == "bwd":
        return sdpa.sdpa_qk_norm_rope_bwd(st["dq_out"], st["dk_out"], st["q"], st["k"], st["cos"],
                                          st["sin"], dv_out=st["dv_out"], **kw)
    if c["way"] == "append":
        kw.update(kv_rows=st["kv_rows"], k_out=st["k_cache"], v_out=st["v_cache"])
    return sdpa.sdpa_qk_norm_rope(st["q"], st["k"], st["cos"], st["sin"], v=st["v"], **kw)


def _cap_own(st):
    import scaled_dot_product_06_gb300 as sdpa
    c = st["case"]
    kw = dict(scale=st["scale"], softcap=c["cap"], window=(c["left"], c["right"]),
              bottom_right=c["bottom_right"])
    q, k, v = st["q"], st["k"], st["v"]
    if c["lens"]:
        pack = (st["starts"], st["starts"], c["s_q"], c["s_kv"])
        o, lse = sdpa.sdpa_fwd_varlen(q, k, v, *pack, **kw)
        if c["way"] == "fwd":
            return o, lse
        return (o, lse, *sdpa.sdpa_bwd_varlen(q, k, v, o, st["do"], lse, *pack, **kw))
    o, lse = sdpa.sdpa_fwd(q, k, v, **kw)
    if c["way"] == "fwd":
        return o, lse
    return (o, lse, *sdpa.sdpa_bwd(q, k, v, o, st["do"], lse, **kw)[:3])


def _prefix_own(st):
    import scaled_dot_product_06_gb300 as sdpa
    c = st["case"]
    return sdpa.sdpa_fwd_prefix(st["q"], st["k_prefix"], st["v_prefix"], st["k"], st["v"], st["lens"],
                                scale=st["scale"], softcap=c["cap"])


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _norm_exact, "cap": _cap_exact, "prefix": _prefix_exact}[case["op"]](st)


def _norm_exact(st):
    c = st["case"]
    half, f64 = c["rot"] // 2, torch.float64
    i = torch.arange(half, device=st["q"].device)
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    # the rotation as a complex product
    turn = torch.complex(st["cos"].to(f64), st["sin"].to(f64))[st["positions"].long()]

    def forward(x, w):  # [b, s, d] of one head
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * w
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first] = z.real
        y[..., second] = z.imag
        return y

    def double(x):
        return None if x is None else x.to(f64)

    qw, kw = double(st["q_weight"]), double(st["k_weight"])
    if c["way"] == "bwd":
        out = []
        for x, dy, w in ((st["q"], st["dq_out"], qw), (st["k"], st["dk_out"], kw)):
            dx, dw = [], 0
            for j in range(x.shape[2]):
                leaves = [x[:, :, j].to(f64).requires_grad_()]
                if w is not None:
                    leaves.append(w.clone().requires_grad_())
                got = torch.autograd.grad(forward(leaves[0], leaves[1] if w is not None else None),
                                          leaves, dy[:, j].to(f64))
                dx.append(got[0])
                dw = dw + got[1] if w is not None else None
            out.append((torch.stack(dx, 2), dw))
        return out[0][0], out[1][0], st["dv_out"].to(f64).transpose(1, 2), out[0][1], out[1][1]
    q = torch.stack([forward(st["q"][:, :, j].to(f64), qw) for j in range(c["h"])], 1)
    k = torch.stack([forward(st["k"][:, :, j].to(f64), kw) for j in range(c["h_kv"])], 1)
    v = st["v"].to(f64).transpose(1, 2)
    if c["way"] == "fwd":
        return q, k, v
    kc, vc = st["k_cache"].to(f64), st["v_cache"].to(f64)
    for j, r in enumerate(st["kv_rows"].tolist()):
        kc[j, :, r:r + c["s"]] = k[j]
        vc[j, :, r:r + c["s"]] = v[j]
    return q, kc, vc


def _attend(q, k, v, cap, scale, hidden):
    """O and LSE of one head in 64 bits; hidden: True where a key is not seen."""
    s = q @ k.transpose(0, 1) * scale
    if cap > 0:
        s = cap * torch.tanh(s / cap)
    s = s.masked_fill(hidden, float("-inf"))
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    return p @ v, lse


def _cap_exact(st):
    c = st["case"]
    f64, grp = torch.float64, c["h"] // c["h_kv"]
    lens, step = c["lens"], c["way"] == "step"
    if lens:
        starts = st["starts"].tolist()
        spans = [(0, starts[i], starts[i + 1]) for i in range(c["b"])]
        q, k, v, do = (st[x][None] for x in ("q", "k", "v", "do"))
    else:
        spans = [(i, 0, None) for i in range(c["b"])]
        q, k, v, do = (st[x] for x in ("q", "k", "v", "do"))
    o = torch.zeros(do.shape, dtype=f64, device=q.device)
    lse = torch.zeros(do.shape[:-1], dtype=f64, device=q.device)
    dq, dk, dv = (torch.zeros(x.shape, dtype=f64, device=q.device) for x in (q, k, v))
    for i, lo, hi in spans:
        for j in range(c["h"]):
            at = (i, j, slice(lo, hi))
            kv = (i, j // grp, slice(lo, hi))
            leaves = [x.to(f64).requires_grad_(step) for x in (q[at], k[kv], v[kv])]
            s_q, s_kv = leaves[0].shape[0], leaves[1].shape[0]
            off = s_kv - s_q if c["bottom_right"] else 0
            place = (torch.arange(s_kv, device=q.device)[None]
                     - torch.arange(s_q, device=q.device)[:, None] - off)
            hidden = torch.zeros_like(place, dtype=torch.bool)
            if c["left"] >= 0:
                hidden |= place < -c["left"]
            if c["right"] >= 0:
                hidden |= place > c["right"]
            # a row that sees nothing is taken out of the sums
            some = ~hidden.all(-1)
            got_o, got_l = _attend(leaves[0][some], leaves[1], leaves[2], c["cap"], st["scale"],
                                   hidden[some])
            o[at][some] = got_o.detach()
            lse[at] = float("-inf")
            lse[at][some] = got_l.detach()
            if step:
                g = torch.autograd.grad(got_o, leaves, do[at][some].to(f64))
                dq[at] += g[0]
                dk[kv] += g[1]
                dv[kv] += g[2]
    out = (o, lse, dq, dk, dv) if step else (o, lse)
    return tuple(x[0] for x in out) if lens else out


def _prefix_exact(st):
    c = st["case"]
    f64, grp, s_q = torch.float64, c["h"] // c["h_kv"], c["s_q"]
    o = torch.zeros(c["b"], c["h"], s_q, c["d_v"], dtype=f64, device=st["q"].device)
    lse = torch.zeros(c["b"], c["h"], s_q, dtype=f64, device=st["q"].device)
    kp, vp = st["k_prefix"].to(f64), st["v_prefix"].to(f64)
    for i, n in enumerate(st["lens"].tolist()):
        place = torch.arange(c["prefix"] + n, device=o.device)[None] - c["prefix"]
        new = torch.arange(s_q, device=o.device)[:, None]
        hidden = (place > n - s_q + new).repeat(grp, 1)
        for j in range(c["h_kv"]):
            k = torch.cat((kp[j], st["k"][i, j, :n].to(f64)))
            v = torch.cat((vp[j], st["v"][i, j, :n].to(f64)))
            q = st["q"][i, j * grp:(j + 1) * grp].to(f64).flatten(0, 1)
            got_o, got_l = _attend(q, k, v, c["cap"], st["scale"], hidden)
            o[i, j * grp:(j + 1) * grp] = got_o.unflatten(0, (grp, s_q))
            lse[i, j * grp:(j + 1) * grp] = got_l.unflatten(0, (grp, s_q))
    return o, lse
