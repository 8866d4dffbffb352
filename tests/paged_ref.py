"""Plain forms of the paged cache for the tests: pages dealt out and slots one
token at a time, attention in fp64 with bounds."""
import numpy as np
import torch

from capped_bounds import u_of


def ceil(a, b):
    return -(-a // b)


def page_slots(lens, new, table, ring, span, page, rows=None, width=None):
    """(slots, positions, starts, lens_out, span_out, table, ring) as lists."""
    table, ring, pool = [list(r) for r in table], list(ring), len(ring)
    head, tail = span
    free = min(max(tail - head, 0), pool)
    wide = len(table[0]) if table else 0
    asked = used = total = returned = 0
    per_request, starts, lens_out = [], [0], []
    back = []
    for i in range(len(lens)):
        n, x = max(lens[i], 0), max(new[i], 0)
        if new[i] < 0:
            back += table[i][:min(ceil(n, page), wide)]
            per_request.append([])
            lens_out.append(0)
            starts.append(starts[-1])
            continue
        k = ceil(n + x, page) - ceil(n, page)
        good = ceil(n + x, page) <= wide and (total + x <= rows if rows is not None else x <= width)
        total += x
        if good:
            asked += k
            good = k == 0 or asked <= free
        if good and k:
            for j in range(k):
                table[i][ceil(n, page) + j] = ring[(head + used + j) % pool]
            used += k
        out = []
        for t in range(x):
            p = n + t
            pg = table[i][p // page] if good else -1
            out.append((pg * page + p % page if 0 <= pg < pool else -1, p))
        per_request.append(out)
        lens_out.append(n + x if good else n)
        starts.append(total if rows is None else min(total, rows))
    for pg in back:
        ring[(tail + returned) % pool] = pg
        returned += 1
    if rows is not None:
        flat = [e for r in per_request for e in r][:rows]
        flat += [(-1, 0)] * (rows - len(flat))
    else:
        flat = [e for r in per_request for e in (r[:width] + [(-1, 0)] * (width - len(r)))]
    return ([e[0] for e in flat], [e[1] for e in flat], starts if rows is not None else None, lens_out,
            [head + used, tail + returned], table, ring)


def f64(t):
    return t.double().cpu().numpy()


def make(b, h, h_kv, s_q, lens, page, d, d_v, t, seed=0, q_mul=3.0, token_major=False, spare=3, junk=-1,
         garbage=True):
    """CPU inputs of sdpa_fwd_paged; what no sequence holds is NaN or infinite."""
    g = torch.Generator().manual_seed(seed)

    def r(*shape, mul=1.0):
        return (torch.randn(*shape, generator=g) * mul).to(t)

    have = [ceil(max(n, 0), page) for n in lens]
    wide, count = max(have + [1]), sum(have) + spare
    order = torch.randperm(count, generator=g).to(torch.int32)
    x = {"q": r(b, h, s_q, d, mul=q_mul), "k_pages": r(count, h_kv, page, d), "v_pages": r(count, h_kv, page, d_v),
         "block_table": torch.full((b, wide + 2), junk, dtype=torch.int32),
         "seqlens_k": torch.tensor(lens, dtype=torch.int32)}
    at = 0
    bad = torch.ones(count, page, dtype=torch.bool)
    for i, n in enumerate(lens):
        x["block_table"][i, :have[i]] = order[at:at + have[i]]
        for c in range(have[i]):
            bad[order[at + c], :min(page, n - c * page)] = False
        at += have[i]
    if garbage:
        x["k_pages"] = x["k_pages"].masked_fill(bad[:, None, :, None], float("nan"))
        x["v_pages"] = x["v_pages"].masked_fill(bad[:, None, :, None], float("nan"))
        x["v_pages"][::2] = x["v_pages"][::2].masked_fill(bad[::2, None, :, None], float("inf"))
    if token_major:
        for n in ("k_pages", "v_pages"):
            x[n] = x[n].transpose(1, 2).contiguous().transpose(1, 2)
    return x


def keys_of(x, i, n, hk, name):
    page = x[name].shape[2]
    ids = x["block_table"][i, :ceil(n, page)].long()
    return f64(x[name][ids, hk].flatten(0, 1)[:n])


def attention(x, scale, cap, left=-1):
    """(o, lse) in fp64 and their bounds: the score's error (fp32 sums of d
    products; capped, softcap 2^-20 more), P and O rounded once each, fp32 sums and
    weights of joined parts within 2^-16 of the sum of absolute values."""
    b, h, s_q, d = x["q"].shape
    h_kv, d_v = x["k_pages"].shape[1], x["v_pages"].shape[3]
    u = u_of(x["q"].dtype)
    sub = 2.0 ** -25 if x["q"].dtype == torch.float16 else 0.0
    o, oe = np.zeros((b, h, s_q, d_v)), np.zeros((b, h, s_q, d_v))
    lse, le = np.full((b, h, s_q), -np.inf), np.zeros((b, h, s_q))
    for i in range(b):
        n = int(x["seqlens_k"][i])
        for hk in range(h_kv):
            k, v = keys_of(x, i, n, hk, "k_pages"), keys_of(x, i, n, hk, "v_pages")
            for j in range(hk * (h // h_kv), (hk + 1) * (h // h_kv)):
                for t in range(s_q):
                    p = n - s_q + t
                    lo = max(0, p - left) if left >= 0 else 0
                    if p + 1 <= lo:
                        continue
                    q, kk, vv = f64(x["q"][i, j, t]), k[lo:p + 1], v[lo:p + 1]
                    s = scale * (kk @ q)
                    es = (abs(scale) * (np.abs(kk) @ np.abs(q)) * d * 2.0 ** -24).max() + cap * 2.0 ** -20
                    if cap:
                        s = cap * np.tanh(s / cap)
                    m = s.max()
                    w = np.exp(s - m)
                    lse[i, j, t] = m + np.log(w.sum())
                    w = w / w.sum()
                    o[i, j, t] = w @ vv
                    oe[i, j, t] = ((u + 2 * es + 2.0 ** -20 + 2.0 ** -16) * w + 256 * sub) @ np.abs(vv) \
                        + u * np.abs(o[i, j, t]) + sub
                    le[i, j, t] = es + 2.0 ** -19 * (1 + abs(lse[i, j, t]) + cap)
    return o, lse, oe, le


def check(x, got, scale, cap=0.0, left=-1):
    from scaled_dot_product_06_gb300 import sdpa_device_error
    torch.cuda.synchronize()
    assert sdpa_device_error() == 0
    o, lse, oe, le = attention(x, scale, cap, left)
    for name, a, r, e in (("o", got[0], o, oe), ("lse", got[1], lse, le)):
        a = f64(a)
        ninf = np.isneginf(r)
        assert np.array_equal(np.isneginf(a), ninf), name
        assert np.isfinite(a[~ninf]).all(), name
        over = np.abs(a[~ninf] - r[~ninf]) - e[~ninf]
        assert over.size == 0 or over.max() <= 0, (
            f"{name}: {int((over > 0).sum())} of {over.size} past their bound by {over.max():.3e}")
