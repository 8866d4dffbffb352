"""What is measured of the paged key/value cache: block tables and slot maps built
from request lengths, the norm, rotation and append of new tokens into pages, and
the attention of the newest tokens over the pages.

``run`` computes a case in plain torch operations (fp32, rounded once at the
end) or, where ``own`` is true, through the package's entry points. ``exact``
computes the same in 64 bits, one sequence and head at a time, and the tables with
whole numbers in plain Python.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# ---------------------------------------------------------------- the cases
def _slots(name, b, page, longest, rows, width, lens, ended=0.0, fresh=False, short=False):
    """b requests of up to `longest` tokens in pages of `page`. rows: packed new
    tokens, `rows` in all (with a padded tail); width: up to `width` new tokens a
    request, padded. ended: share of requests that have ended; fresh: all begin with
    this call; short: there are fewer free pages than asked for."""
    return {"name": name, "op": "slots", "b": b, "page": page, "longest": longest, "rows": rows,
            "width": width, "lens": lens, "ended": ended, "fresh": fresh, "short": short}


def _append(name, b, s, h, h_kv, d, d_v, dtype, rot, page, lens, interleaved=False, normed=True,
            token_major=False):
    """s new tokens of each of b rows into pages; some slots are -1 (padding)."""
    return {"name": name, "op": "append", "b": b, "s": s, "h": h, "h_kv": h_kv, "d": d, "d_v": d_v,
            "dtype": dtype, "rot": rot, "page": page, "lens": lens, "interleaved": interleaved,
            "normed": normed, "token_major": token_major}


def _paged(name, b, h, h_kv, s_q, d, d_v, dtype, page, longest, lens, shortest=0, cap=0.0, left=-1,
           token_major=False):
    """s_q newest tokens of b sequences of shortest to longest keys; token_major: the
    pages hold [page][h_kv][d] rather than [h_kv][page][d]."""
    return {"name": name, "op": "paged", "b": b, "h": h, "h_kv": h_kv, "s_q": s_q, "d": d, "d_v": d_v,
            "dtype": dtype, "page": page, "longest": longest, "lens": lens, "shortest": shortest,
            "cap": cap, "left": left, "token_major": token_major}


def listed():
    return [
        # the tables of one decoding step of a large batch, a few of its requests ended
        _slots("slots-decode-b256", 256, 16, 4096, 0, 1, 1, ended=0.05),
        # prompts that have just arrived, packed, in large pages
        _slots("slots-prompts-t16384", 13, 64, 2048, 16384, 0, 2, fresh=True),
        # a mixed step of many requests: decoding ones, pieces of prompts, ended ones
        _slots("slots-mixed-b1000", 1000, 16, 2048, 131072, 0, 3, ended=0.1),
        # one decoding step: norm, rotate and append one token of each sequence
        _append("append-decode-b256", 256, 1, 32, 4, 128, 128, "bf16", 128, 16, 1),
        # packed prompts with a padded tail, wide heads turned in part
        _append("append-prompts-t8191", 1, 8191, 16, 4, 192, 128, "fp16", 64, 64, 2, interleaved=True),
        # the smallest call, where latency counts: two sequences just begun
        _paged("paged-b2-n17-d64", 2, 8, 1, 1, 64, 64, "bf16", 16, 17, 1),
        # one user with a long context
        _paged("paged-b1-n131072", 1, 32, 8, 1, 128, 128, "bf16", 64, 131072, 2, shortest=131071),
        # a served batch of ragged lengths in small pages
        _paged("paged-b64-n8192", 64, 32, 4, 1, 128, 128, "bf16", 16, 8192, 3),
        # a large batch of short conversations, one K/V head a query head
        _paged("paged-b256-n777-mha", 256, 16, 16, 1, 128, 128, "fp16", 32, 777, 4),
        # all query heads on one K/V head, wide heads, capped scores
        _paged("paged-mqa-d192-cap50", 96, 16, 1, 1, 192, 128, "bf16", 64, 5000, 5, cap=50.0),
        # four drafted tokens at a time under a sliding window, token-major pages
        _paged("paged-draft4-window4096", 16, 32, 8, 4, 128, 128, "bf16", 128, 16384, 6, shortest=2000,
               left=4096, token_major=True),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_once(rng):
    op = rng.choice(("slots", "append", "paged", "paged"))
    page = rng.choice((16, 32, 64, 128, 256))
    lens = rng.randrange(1, 100000)
    if op == "slots":
        b = _log(rng, 1, 1000)
        longest = _log(rng, 1, 8192)
        packed = rng.random() < 0.5
        return _slots(None, b, page, longest, _log(rng, 1, 131072) if packed else 0,
                      0 if packed else _log(rng, 1, min(64, 131072 // b)), lens,
                      ended=rng.choice((0.0, 0.1, 0.3)), fresh=rng.random() < 0.2,
                      short=rng.random() < 0.2)
    dtype = rng.choice(("bf16", "fp16"))
    d, d_v = rng.choice(((64, 64), (128, 128), (192, 128)))
    h_kv = rng.choice((1, 2, 3, 4, 8, 16))
    h = h_kv * rng.choice((1, 2, 4, 5, 8))
    if op == "append":
        return _append(None, _log(rng, 1, 256), _log(rng, 1, 4096), h, h_kv, d, d_v, dtype,
                       rng.choice((16, 32, 48, 64, d)), page, lens, rng.random() < 0.4,
                       rng.random() < 0.8, rng.random() < 0.5)
    longest = _log(rng, 1, 131072)
    return _paged(None, _log(rng, 1, 256), h, h_kv, rng.choice((1, 1, 1, 1, 2, 3, 4, 8)), d, d_v, dtype, page,
                  longest, lens, rng.choice((0, 0, longest // 2)), rng.choice((0.0, 0.0, 20.0, 50.0)),
                  rng.choice((-1, -1, -1, _log(rng, 16, 8192))), rng.random() < 0.4)


def draw(rng):
    most, width = {}, 0
    for c in listed():
        w = work(c)
        for k in ("bytes", "flops"):
            most[c["op"], k] = max(most.get((c["op"], k), 0), w[k])
        width = max(width, _gathered(c))
    while True:
        c = _draw_once(rng)
        c.pop("name")
        w = work(c)
        if _gathered(c) <= width and all(w[k] <= most[c["op"], k] for k in w):
            return c


def _gathered(c):
    """Elements that the plain form gathers and the scores that it holds."""
    if c["op"] != "paged":
        return 0
    return c["b"] * c["longest"] * (c["h_kv"] * (c["d"] + c["d_v"]) + 4 * c["h"] * c["s_q"])


def _lengths(c):
    """Keys of each sequence, the new tokens' among them; one has the longest."""
    rng = random.Random(c["lens"])
    n = [rng.randrange(c["shortest"], c["longest"] + 1) for _ in range(c["b"])]
    n[rng.randrange(c["b"])] = c["longest"]
    return n


def _requests(c):
    """(tokens in the cache, new ones or -1) of each request, and the free pages."""
    rng = random.Random(c["lens"])
    n = [0 if c["fresh"] else rng.randrange(0, c["longest"] + 1) for _ in range(c["b"])]
    new, left = [], c["rows"]
    for i in range(c["b"]):
        if rng.random() < c["ended"]:
            new.append(-1)
        elif c["width"]:
            new.append(rng.randrange(1 if c["width"] == 1 else 0, c["width"] + 1))
        else:
            # decoding requests, idle ones, and prompts or pieces of them
            most = (2 if c["fresh"] else 8) * c["rows"] // c["b"]
            some = rng.randrange(1, max(2, min(c["longest"], most) + 1))
            t = some if c["fresh"] else rng.choice((0, 1, 1, some))
            t = min(t, left)
            left -= t
            new.append(t)
    asked = sum(_pages(x + max(y, 0), c["page"]) - _pages(x, c["page"]) for x, y in zip(n, new))
    free = rng.randrange(asked // 2, asked + 1) if c["short"] else asked + rng.randrange(1, 100)
    return n, new, free


def _pages(tokens, page):
    return (tokens + page - 1) // page


def work(case):
    c = case
    if c["op"] == "slots":
        n, new, free = _requests(c)
        rows = c["rows"] or c["b"] * c["width"]
        grown = sum(_pages(x + max(y, 0), c["page"]) - _pages(x, c["page"]) for x, y in zip(n, new))
        back = sum(_pages(x, c["page"]) for x, y in zip(n, new) if y < 0)
        partial = sum(1 for x, y in zip(n, new) if y > 0 and x % c["page"])
        return {"bytes": 12 * c["b"] + 32 + 8 * rows + 8 * min(grown, free) + 8 * back + 4 * partial
                + (4 * (c["b"] + 1) if c["rows"] else 0), "flops": 0}
    d, d_v = c["d"], c["d_v"]
    if c["op"] == "append":
        tok = c["b"] * c["s"]
        turned = tok * (c["h"] + c["h_kv"]) * d
        el = turned + tok * c["h_kv"] * d_v
        return {"bytes": 2 * 2 * el + 4 * tok * (c["rot"] + 2), "flops": 10 * turned}
    pairs = keys = pages = 0
    for n in _lengths(c):
        seen = [_span(c, n, t) for t in range(c["s_q"])]
        pairs += sum(max(0, hi - lo) for lo, hi in seen)
        lo, hi = min(x for x, _ in seen), max(0, max(x for _, x in seen))
        keys += max(0, hi - lo)
        pages += _pages(hi, c["page"]) - lo // c["page"] if hi > lo else 0
    rows = c["b"] * c["h"] * c["s_q"]
    return {"bytes": 2 * (d + d_v) * (c["h_kv"] * keys + rows) + 4 * rows + 4 * pages + 4 * c["b"],
            "flops": 2 * (d + d_v) * pairs * c["h"]}


def _span(c, n, t):
    """Keys [lo, hi) that new token t of a sequence of n keys sees."""
    last = n - c["s_q"] + t
    return (max(0, last - c["left"]) if c["left"] >= 0 else 0), last + 1


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    st = {"case": dict(c)}

    def ints(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device=dev)

    if c["op"] == "slots":
        n, new, free = _requests(c)
        have = [_pages(x, c["page"]) for x in n]
        # (some requests may ask for more than their row of the table holds)
        st["wide"] = max(1, _pages(c["longest"] + (c["width"] or c["longest"]), c["page"]))
        pool = max(1, sum(have) + free)
        order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
        st["block_table"] = torch.full((c["b"], st["wide"]), -1, dtype=torch.int32, device=dev)
        owned = torch.arange(st["wide"], device=dev)[None] < ints(have)[:, None]
        st["block_table"][owned] = order[:sum(have)]
        # the ring has turned a few times
        head = int(seed) % 7 * pool + pool // 3
        st["free_pages"] = order.clone()
        at = (head + torch.arange(free, device=dev)) % pool
        st["free_pages"][at] = order[sum(have):sum(have) + free]
        st["free_range"] = ints([head, head + free], torch.int64)
        st["seqlens"], st["new_tokens"] = ints(n), ints(new)
        return st

    t = DTYPES[c["dtype"]]

    def randn(*shape, mul=1.0, dtype=t):
        return (torch.randn(*shape, generator=g, device=dev) * mul).to(dtype)

    h, h_kv, d, d_v, page = (c[k] for k in ("h", "h_kv", "d", "d_v", "page"))

    def pages(count, width):
        if c["token_major"]:
            return randn(count, page, h_kv, width).transpose(1, 2)
        return randn(count, h_kv, page, width)

    if c["op"] == "append":
        b, s, rot = c["b"], c["s"], c["rot"]
        qkv = randn(b, s, h * d + h_kv * (d + d_v), mul=2.0)  # the fused projection's output
        st["q"] = qkv[..., :h * d].unflatten(-1, (h, d))
        st["k"] = qkv[..., h * d:(h + h_kv) * d].unflatten(-1, (h_kv, d))
        st["v"] = qkv[..., (h + h_kv) * d:].unflatten(-1, (h_kv, d_v))
        st["q_weight"] = st["k_weight"] = None
        if c["normed"]:
            st["q_weight"] = 1.0 + randn(d, mul=0.1, dtype=torch.float32)
            st["k_weight"] = 1.0 + randn(d, mul=0.1, dtype=torch.float32)
        base = torch.randint(0, 30000, (b, 1), generator=g, device=dev)
        st["positions"] = (base + torch.arange(s, device=dev)).to(torch.int32)
        n_pos = 30000 + s
        inv = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=dev),
                        -torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
        ang = torch.arange(n_pos, dtype=torch.float64, device=dev)[:, None] * inv
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        # each row's tokens lie one after another from some place in its first page
        first = torch.randint(0, page, (b, 1), generator=g, device=dev)
        wide = _pages(page - 1 + s, page)
        count = b * wide + 3
        table = torch.randperm(count, generator=g, device=dev)[:b * wide].view(b, wide)
        at = first + torch.arange(s, device=dev)
        slots = table.gather(1, at // page) * page + at % page
        rng = random.Random(c["lens"])
        tail = s - rng.randrange(0, s // 16 + 1)
        slots[:, tail:] = -1  # padding
        if s == 1 and b > 8:
            slots[rng.randrange(b)] = -1  # an idle request
        st["kv_slots"] = slots.to(torch.int32).contiguous()
        st["k_pages"], st["v_pages"] = pages(count, d), pages(count, d_v)
        return st

    n, s_q, b = _lengths(c), c["s_q"], c["b"]
    wide = _pages(c["longest"], page)
    have = [_pages(x, page) for x in n]
    count = sum(have) + 5
    order = torch.randperm(count, generator=g, device=dev)
    st["seqlens_k"] = ints(n)
    owned = torch.arange(wide, device=dev)[None] < ints(have)[:, None]
    st["block_table"] = torch.full((b, wide), -1, dtype=torch.int32, device=dev)
    st["block_table"][owned] = order[:sum(have)].to(torch.int32)
    st["q"] = randn(b, h, s_q, d, mul=2.0)
    st["k_pages"], st["v_pages"] = pages(count, d), pages(count, d_v)
    # what nobody has, and what lies behind a sequence's last token in its last page, is
    # whatever was there before
    st["k_pages"][order[sum(have):]] = float("nan")
    st["v_pages"][order[sum(have):]] = float("nan")
    live = st["seqlens_k"] > 0
    last = st["block_table"].long().gather(1, (st["seqlens_k"].long()[:, None] - 1).clamp(min=0) // page)
    behind = torch.arange(page, device=dev)[None] >= ((st["seqlens_k"][:, None] - 1) % page + 1)
    for x in (st["k_pages"], st["v_pages"]):
        rows = x[last[live, 0]]
        x[last[live, 0]] = rows.masked_fill(behind[live][:, None, :, None], float("nan"))
    st["scale"] = 1.0 / math.sqrt(d)
    return st


# ---------------------------------------------------------------- plain forms
def _slots_plain(st):
    c = st["case"]
    page, wide, b = c["page"], st["wide"], c["b"]
    table, ring, span = st["block_table"], st["free_pages"], st["free_range"]
    pool, dev = ring.numel(), table.device
    n, new = st["seqlens"].long().clamp(min=0), st["new_tokens"].long()
    ended, add = new < 0, new.clamp(min=0)
    have = torch.div(n + page - 1, page, rounding_mode="floor")
    need = torch.div(n + add + page - 1, page, rounding_mode="floor")
    ends = add.cumsum(0)
    fits = ~ended & (need <= wide) & ((ends <= c["rows"]) if c["rows"] else (add <= c["width"]))
    take = torch.where(fits, need - have, 0)
    upto = take.cumsum(0)
    served = fits & ((take == 0) | (upto <= (span[1] - span[0]).clamp(0, pool)))
    n_out = torch.where(ended, 0, torch.where(served, n + add, n))
    back = torch.where(ended, have.clamp(max=wide), 0)
    col = torch.arange(wide, device=dev)[None]
    fresh = served[:, None] & (col >= have[:, None]) & (col < need[:, None])
    given = ring[(span[0] + (upto - take)[:, None] + col - have[:, None]) % pool]
    # the pages that come back, each to its place behind the ring's end
    gone = (span[1] + (back.cumsum(0) - back)[:, None] + col) % pool
    keep = torch.cat((ring, ring.new_zeros(1)))
    keep[torch.where(col < back[:, None], gone, pool)] = table
    table.copy_(torch.where(fresh, given, table))
    ring.copy_(keep[:pool])
    if c["rows"]:
        r = torch.arange(c["rows"], device=dev)
        i = torch.searchsorted(ends, r, right=True)
        there = i < b
        i = i.clamp(max=b - 1)
        t = r - (ends - add)[i]
    else:
        i = torch.arange(b, device=dev)[:, None].expand(b, c["width"])
        t = torch.arange(c["width"], device=dev)[None].expand(b, c["width"])
        there = t < add[:, None]
    pos = n[i] + t
    at = torch.div(pos, page, rounding_mode="floor").clamp(0, wide - 1)
    pg = table[i, at].long()
    ok = there & served[i] & (pg >= 0) & (pg < pool)
    out = [torch.where(ok, pg * page + pos % page, -1).to(torch.int32), torch.where(there, pos, 0).to(torch.int32)]
    if c["rows"]:
        out.append(torch.cat((ends.new_zeros(1), ends)).clamp(max=c["rows"]).to(torch.int32))
    taken = torch.where(served, take, 0).sum()
    return (*out, n_out.to(torch.int32), torch.stack((span[0] + taken, span[1] + back.sum())), table, ring)


def _rotate(x, cos, sin, rot, interleaved):
    """The first `rot` elements of x's last dimension rotated; cos, sin broadcast to x."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _append_plain(st):
    c = st["case"]
    t, rot, page = DTYPES[c["dtype"]], c["rot"], c["page"]
    pos = st["positions"].long()
    cos, sin = st["cos"][pos][:, :, None], st["sin"][pos][:, :, None]  # [b, s, 1, rot / 2]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        return _rotate(x, cos, sin, rot, c["interleaved"]).to(t)

    q, k = turned(st["q"], st["q_weight"]), turned(st["k"], st["k_weight"])
    slots = st["kv_slots"].long()
    some = slots >= 0
    pg, row = slots[some] // page, slots[some] % page
    st["k_pages"][pg, :, row] = k[some]
    st["v_pages"][pg, :, row] = st["v"][some]
    return q.transpose(1, 2).contiguous(), st["k_pages"], st["v_pages"]


def _paged_plain(st):
    c = st["case"]
    t, s_q, grp = DTYPES[c["dtype"]], c["s_q"], c["h"] // c["h_kv"]
    n, table = st["seqlens_k"].long(), st["block_table"].long().clamp(min=0)
    q = st["q"].float().unflatten(1, (c["h_kv"], grp)).flatten(2, 3)  # [b, h_kv, group * s_q, d]
    at = torch.arange(table.shape[1] * c["page"], device=q.device)
    behind = (at >= n[:, None])[:, None, :, None]

    def gathered(pages):  # [b, h_kv, keys, width]
        x = pages[table].transpose(1, 2).flatten(2, 3).float()
        return x.masked_fill_(behind, 0.0)

    s = torch.matmul(q, gathered(st["k_pages"]).mT) * st["scale"]
    if c["cap"] > 0:
        s = torch.tanh(s / c["cap"]) * c["cap"]
    # new token i of a sequence sees the keys up to its own place
    last = (n[:, None] - s_q + torch.arange(s_q, device=q.device))[:, :, None]
    seen = at <= last
    if c["left"] >= 0:
        seen &= at >= last - c["left"]
    s = s.masked_fill_(~seen[:, None].repeat(1, 1, grp, 1), float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    o = torch.matmul(p, gathered(st["v_pages"]))
    o = o.unflatten(2, (grp, s_q)).flatten(1, 2).to(t)
    return o, (m + torch.log(total)).squeeze(-1).unflatten(2, (grp, s_q)).flatten(1, 2)


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"slots": _slots_own, "append": _append_own, "paged": _paged_own}[op](state)
    return {"slots": _slots_plain, "append": _append_plain, "paged": _paged_plain}[op](state)


def _slots_own(st):
    import scaled_dot_product_06_gb300 as sdpa
    c = st["case"]
    tokens = {"rows": c["rows"]} if c["rows"] else {"width": c["width"]}
    out = sdpa.sdpa_page_slots(st["seqlens"], st["new_tokens"], st["block_table"], st["free_pages"],
                               st["free_range"], c["page"], **tokens)
    return (*(x for x in out if x is not None), st["block_table"], st["free_pages"])


def _append_own(st):
    import scaled_dot_product_06_gb300 as sdpa
    c = st["case"]
    return sdpa.sdpa_qk_norm_rope(st["q"], st["k"], st["cos"], st["sin"], v=st["v"], positions=st["positions"],
                                  q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS,
                                  interleaved=c["interleaved"], kv_slots=st["kv_slots"], k_out=st["k_pages"],
                                  v_out=st["v_pages"])


def _paged_own(st):
    import scaled_dot_product_06_gb300 as sdpa
    c = st["case"]
    return sdpa.sdpa_fwd_paged(st["q"], st["k_pages"], st["v_pages"], st["block_table"], st["seqlens_k"],
                               scale=st["scale"], softcap=c["cap"], window_left=c["left"])


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"slots": _slots_exact, "append": _append_exact, "paged": _paged_exact}[case["op"]](st)


def _slots_exact(st):
    c = st["case"]
    page, wide, rows = c["page"], st["wide"], c["rows"]
    table, ring = st["block_table"].tolist(), st["free_pages"].tolist()
    head, tail = st["free_range"].tolist()
    pool, given, want = len(ring), min(max(tail - head, 0), len(ring)), 0
    slots, places, starts, n_out, back = [], [], [0], [], []
    total = taken = 0
    for i, (n, new) in enumerate(zip(st["seqlens"].tolist(), st["new_tokens"].tolist())):
        have, count = _pages(n, page), max(new, 0)
        if new < 0:
            back += table[i][:have]
            n_out.append(0)
            ok = False
        else:
            grown = _pages(n + new, page) - have
            ok = have + grown <= wide and (total + new <= rows if rows else new <= c["width"])
            if ok:
                begin, want = want, want + grown
                ok = grown == 0 or want <= given
                if ok:
                    taken += grown
                    for j in range(grown):
                        table[i][have + j] = ring[(head + begin + j) % pool]
            n_out.append(n + new if ok else n)
        for t in range(count if rows else c["width"]):
            if rows and total + t >= rows:
                break
            p = n + t
            places.append(p if t < count else 0)
            slots.append(table[i][p // page] * page + p % page if ok and t < count else -1)
        total += count
        starts.append(min(total, rows))
    for j, pg in enumerate(back):
        ring[(tail + j) % pool] = pg
    if rows:
        slots += [-1] * (rows - len(slots))
        places += [0] * (rows - len(places))
    dev = st["seqlens"].device

    def ints(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device=dev)

    shape = (rows,) if rows else (c["b"], c["width"])
    out = [ints(slots).view(shape), ints(places).view(shape)] + ([ints(starts)] if rows else [])
    return (*out, ints(n_out), ints([head + taken, tail + len(back)], torch.int64), ints(table), ints(ring))


def _append_exact(st):
    c = st["case"]
    half, f64, page = c["rot"] // 2, torch.float64, c["page"]
    i = torch.arange(half, device=st["q"].device)
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    # the rotation as a complex product
    turn = torch.complex(st["cos"].to(f64), st["sin"].to(f64))[st["positions"].long()]

    def forward(x, w):  # [b, s, d] of one head
        x = x.to(f64)
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * w.to(f64)
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first] = z.real
        y[..., second] = z.imag
        return y

    q = torch.stack([forward(st["q"][:, :, j], st["q_weight"]) for j in range(c["h"])], 1)
    kc, vc = st["k_pages"].to(f64), st["v_pages"].to(f64)
    slots = st["kv_slots"].long().flatten()
    at = torch.nonzero(slots >= 0).flatten()
    for j in range(c["h_kv"]):
        kc[slots[at] // page, j, slots[at] % page] = forward(st["k"][:, :, j], st["k_weight"]).flatten(0, 1)[at]
        vc[slots[at] // page, j, slots[at] % page] = st["v"][:, :, j].to(f64).flatten(0, 1)[at]
    return q, kc, vc


def _paged_exact(st):
    c = st["case"]
    f64, grp, s_q = torch.float64, c["h"] // c["h_kv"], c["s_q"]
    dev = st["q"].device
    o = torch.zeros(c["b"], c["h"], s_q, c["d_v"], dtype=f64, device=dev)
    lse = torch.full((c["b"], c["h"], s_q), float("-inf"), dtype=f64, device=dev)
    for i, n in enumerate(st["seqlens_k"].tolist()):
        ids = st["block_table"][i, :_pages(n, c["page"])].long()
        k = st["k_pages"][ids].transpose(0, 1).flatten(1, 2)[:, :n]
        v = st["v_pages"][ids].transpose(0, 1).flatten(1, 2)[:, :n]
        for t in range(s_q):
            lo, hi = _span(c, n, t)
            if hi <= lo:
                continue
            for j in range(c["h_kv"]):
                heads = slice(j * grp, (j + 1) * grp)
                s = st["q"][i, heads, t].to(f64) @ k[j, lo:hi].to(f64).T * st["scale"]
                if c["cap"] > 0:
                    s = c["cap"] * torch.tanh(s / c["cap"])
                lse[i, heads, t] = torch.logsumexp(s, -1)
                o[i, heads, t] = torch.softmax(s, -1) @ v[j, lo:hi].to(f64)
    return o, lse
