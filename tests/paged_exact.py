"""Inputs and bounds for the attention over a paged cache that leave room for its
own roundings only: dot products that are exact in fp32, and values whose weighted
sum nearly cancels, so that O's own rounding hides nothing.

With u = finfo(dtype).eps / 2, weights w (they sum to 1) and scores s of a row:

* q and k are multiples of 1/16 of at most 2 in magnitude: products of them are
  multiples of 2^-8 of at most 4, their sums over d <= 192 stay below 2^10: exact in
  fp32, in any order.
* The factor of the exponent is rounded twice (2^-23 of it), and the exponent itself
  once; with |s log2 e| below 32 that moves P by 32 ln 2 (2^-23 + 2^-24) < 2^-17.4 at
  its far end, and by |s| (2^-23 + 2^-24) at s; the row's sum by as much again at
  most, so 2 |s|max 2^-22. The exponential: 2^-22, twice.
* P in two 16-bit parts: the low one rounds what the high one left, u^2 of P.
* Sums in fp32: a step of 16 keys adds once to O, cut off at 2^-23 of it; the sum of
  P, the factors at a unit's end and the join of parts add sixteen roundings more.
* O is rounded once: u of it, in fp16 2^-25 where it is small.
"""
import numpy as np
import torch

from capped_bounds import u_of


def grid(shape, g, most=2.0):
    """Multiples of 1/16 of at most `most` in magnitude."""
    return torch.randint(-int(16 * most), int(16 * most) + 1, shape, generator=g).float() / 16


def signs(w, rng):
    """Signs of weights [..., n] whose signed sum is small: the first ones in any order
    by chance, the others, the largest first, each against what has gathered so far."""
    n = w.shape[-1]
    order = rng.permutation(n)
    free = np.broadcast_to(order[:n // 8], w.shape[:-1] + (n // 8,))
    rest = order[n // 8:]
    order = np.concatenate((free, rest[np.argsort(-w[..., rest], axis=-1)]), -1)
    out, total = np.zeros_like(w), np.zeros(w.shape[:-1])
    for j in range(n):
        at = order[..., j:j + 1]
        s = np.where(rng.random(total.shape) < 0.5 if j < n // 8 else total > 0, -1.0, 1.0)
        np.put_along_axis(out, at, s[..., None], -1)
        total += s * np.take_along_axis(w, at, -1)[..., 0]
    return out


def weights(q, k, scale):
    """(scores, weights) of rows q [..., r, d] over keys k [..., n, d], fp64."""
    s = scale * (q.double().numpy() @ np.swapaxes(k.double().numpy(), -1, -2))
    w = np.exp(s - s.max(-1, keepdims=True))
    return s, w / w.sum(-1, keepdims=True)


def cancelling(h_kv, r, n, d, d_v, t, seed):
    """(q [h_kv, r, d], k [h_kv, n, d], v [h_kv, n, d_v]) of one sequence: column c of the
    values nearly cancels for row c mod r, and has magnitudes of its own (powers of
    two, so that a value is exact in either type)."""
    g = torch.Generator().manual_seed(seed)
    q, k = grid((h_kv, r, d), g, 1.0), grid((h_kv, n, d), g, 1.0)
    _, w = weights(q, k, d ** -0.5)
    v, rng = np.zeros((h_kv, n, d_v)), np.random.default_rng(seed)
    for c in range(d_v):
        v[:, :, c] = signs(w[:, c % r], rng) * 2.0 ** (c % 5 - 2)
    return q.to(t), k.to(t), torch.from_numpy(v).to(t)


def bounds(s, w, v, t):
    """(o, lse, bounds) of fp64 scores, weights [..., r, n] and values [..., n, d_v]."""
    u, n = u_of(t), s.shape[-1]
    o = w @ v
    top = np.abs(s).max(-1)
    rel = 2 * top * 2.0 ** -22 + 2.0 ** -21 + u * u + (n / 16 + 16) * 2.0 ** -23
    sub = 2.0 ** -25 if t == torch.float16 else 0.0
    oe = rel[..., None] * (w @ np.abs(v)) + u * np.abs(o) + sub
    m = s.max(-1)
    lse = m + np.log(np.exp(s - m[..., None]).sum(-1))
    # the logarithm: 2^-21 of the type's unit, and two roundings of a number of its size
    le = 2 * top * 2.0 ** -22 + 2.0 ** -20 + (n / 128 + 16) * 2.0 ** -24 + np.abs(lse) * 2.0 ** -21
    return o, lse, oe, le


def paged(q, k, v, page, seed=0):
    """Arguments of sdpa_fwd_paged for sequences q [b, h, 1, d], k, v [b][h_kv, n, d], CPU."""
    count = sum(-(-x.shape[1] // page) for x in k)
    wide = max(-(-x.shape[1] // page) for x in k)
    order = torch.randperm(count, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    h_kv = k[0].shape[0]
    kp = torch.zeros(count, h_kv, page, k[0].shape[2], dtype=q.dtype)
    vp = torch.zeros(count, h_kv, page, v[0].shape[2], dtype=q.dtype)
    table, at = torch.zeros(len(k), wide, dtype=torch.int32), 0
    for i, (a, b) in enumerate(zip(k, v)):
        for c in range(-(-a.shape[1] // page)):
            pg = int(order[at])
            table[i, c] = pg
            at += 1
            part = slice(c * page, min((c + 1) * page, a.shape[1]))
            kp[pg, :, :part.stop - part.start] = a[:, part]
            vp[pg, :, :part.stop - part.start] = b[:, part]
    return {"q": q, "k_pages": kp, "v_pages": vp, "block_table": table,
            "seqlens_k": torch.tensor([x.shape[1] for x in k], dtype=torch.int32)}
