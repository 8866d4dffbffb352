"""What the attention over a paged cache states of its precision: O within its own
rounding where sums cancel, P in two parts, capped scores to the finer tanh; bounds in
paged_exact, and that a coarser form is outside them in test_paged_bounds."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from capped_bounds import u_of
from paged_exact import bounds, cancelling, grid, paged, weights
from paged_ref import attention, check, f64, make
from scaled_dot_product_06_gb300 import sdpa_device_error, sdpa_fwd_paged, sdpa_fwd_prefix
from scaled_dot_product_06_gb300.inputs import DTYPES
from test_paged_bounds import capped_bound

pytestmark = pytest.mark.gpu


def call(x, **kw):
    got = sdpa_fwd_paged(**{n: t.cuda() for n, t in x.items()}, **kw)
    torch.cuda.synchronize()
    assert sdpa_device_error() == 0
    return got


def within(name, got, want, err):
    over = np.abs(f64(got) - want) - err
    assert over.max() <= 0, f"{name}: {int((over > 0).sum())} of {over.size} past their bound by {over.max():.3e}"


# (h_kv, rows a K/V head, lengths, d, d_v): all row blocks (8, 16, 32, 64, two of 64); whole and cut
EXACT = [
    (2, 8, [64, 100, 33, 128], 64, 64),
    (1, 3, [1, 2, 129, 640], 128, 128),
    (2, 16, [100, 64, 200], 192, 128),
    (1, 32, [64, 700], 128, 128),
    (1, 64, [96, 300], 64, 64),
    (1, 64, [64], 192, 128),
    (1, 96, [64, 600], 64, 64),
    (3, 4, [3000, 64, 900, 1500], 128, 128),
    (1, 16, [20000], 64, 64),
]


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("c", EXACT, ids=lambda c: f"kv{c[0]}r{c[1]}n{max(c[2])}d{c[3]}")
def test_only_the_roundings_of_o_are_left(c, t):
    h_kv, r, lens, d, d_v = c
    seqs = [cancelling(h_kv, r, n, d, d_v, DTYPES[t], seed=n + r) for n in lens]
    q = torch.stack([s[0].flatten(0, 1) for s in seqs])[:, :, None]
    got = call(paged(q, [s[1] for s in seqs], [s[2] for s in seqs], 16))
    for i, (qi, ki, vi) in enumerate(seqs):
        s, w = weights(qi, ki, d ** -0.5)
        o, lse, oe, le = bounds(s, w, vi.double().numpy(), DTYPES[t])
        within("o", got[0][i, :, 0], o.reshape(-1, d_v), oe.reshape(-1, d_v))
        within("lse", got[1][i, :, 0], lse.reshape(-1), le.reshape(-1))


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("cap", [50.0, 1000.0])
def test_capped_scores_of_single_keys(t, cap):
    """Sequences of one key: LSE is the capped score, O the value."""
    b, h, d = 300, 8, 64
    g = torch.Generator().manual_seed(3)
    q, k, v = grid((b, h, 1, d), g, 1.5).to(DTYPES[t]), grid((b, 1, 1, d), g, 1.5).to(DTYPES[t]), grid((b, 1, 1, d), g)
    o, lse = call(paged(q, list(k), list(v.to(DTYPES[t])), 16), softcap=cap, scale=0.125)
    s = 0.125 * (f64(q) @ np.swapaxes(f64(k), -1, -2))[..., 0]
    assert np.abs(s).max() > 1
    within("lse", lse, cap * np.tanh(s / cap), capped_bound(s, cap))
    assert torch.equal(o.cpu(), v.to(DTYPES[t]).expand(b, h, 1, d))


@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_the_same_keys_in_a_contiguous_cache(t):
    """O and LSE of both operators over the same keys, element by element: each O is
    rounded once, and the other operator's P is."""
    lens, dt = [900, 1, 333, 512], DTYPES[t]
    x = make(4, 16, 4, 1, lens, 16, 128, 128, dt)
    k, v = torch.zeros(4, 4, 900, 128).to(dt), torch.zeros(4, 4, 900, 128).to(dt)
    for i, n in enumerate(lens):
        for name, c in (("k_pages", k), ("v_pages", v)):
            ids = x["block_table"][i, :(n + 15) // 16].long()
            c[i, :, :n] = x[name][ids].transpose(0, 1).flatten(1, 2)[:, :n]
    e = torch.zeros(4, 0, 128).to(dt).cuda()
    o, lse = sdpa_fwd_prefix(x["q"].cuda(), e, e, k.cuda(), v.cuda(), x["seqlens_k"].cuda())
    got = call(x)
    scale = 128 ** -0.5
    check(x, got, scale)
    # of each row: w @ |v|, and how far an fp32 score may be off
    mag = attention({**x, "v_pages": x["v_pages"].abs()}, scale, 0.0)[0]
    es = np.zeros(mag.shape[:3])
    for i, n in enumerate(lens):
        kk = np.abs(f64(k[i, :, :n])).repeat(4, 0)
        es[i, :, 0] = scale * (kk @ np.abs(f64(x["q"][i, :, 0]))[:, :, None]).max((1, 2)) * 128 * 2.0 ** -24
    u, sub = u_of(dt), 2.0 ** -25 if t == "fp16" else 0.0
    # the other operator's P: u, in fp16 2^-25 of the largest a key; of both: scores, sums in fp32, O
    err = (u + 4 * es[..., None] + 2.0 ** -15) * mag + u * (np.abs(f64(o)) + np.abs(f64(got[0]))) \
        + sub * (2 + np.abs(f64(v)).sum(2).max())
    within("o", got[0], f64(o), err)
    within("lse", got[1], f64(lse), 2 * es + 2.0 ** -18 * (1 + np.abs(f64(lse))))
