"""Calls at the far ends of what the norm, capped and shared-prefix operators take:
caches whose offsets pass 32 bits, many new tokens at a time, rows that belong to no
sequence. Reference: plain torch in fp64 on the device, with the bounds that each
operator's own tests derive (here as one figure: P and O rounded once each, u of sum
P |V|, twice that and an absolute 2^-16 for the fp32 sums).
"""
from __future__ import annotations

import pytest
import torch

from scaled_dot_product_06_gb300 import (sdpa_bwd_varlen, sdpa_device_error, sdpa_fwd_prefix, sdpa_fwd_varlen,
                                         sdpa_qk_norm_rope)

pytestmark = pytest.mark.gpu

U = 2.0 ** -8  # a bf16 rounding


def attend(q, k, v, visible, scale, cap):
    """O, LSE and sum P |V| of one sequence and head; visible [rows, keys]."""
    s = scale * (q.double() @ k.double().T)
    if cap:
        s = cap * torch.tanh(s / cap)
    s = s.masked_fill(~visible, float("-inf"))
    p = torch.softmax(s, -1)
    return p @ v.double(), torch.logsumexp(s, -1), p @ v.double().abs()


def close(o, lse, ref, cap=0.0):
    e = 2 * cap * 2.0 ** -20 + 2.0 ** -16
    assert ((o.double() - ref[0]).abs() <= (2 * U + 4 * e) * ref[2] + 2.0 ** -16).all()
    assert ((lse.double() - ref[1]).abs() <= e * (1 + ref[1].abs())).all()


def test_cache_past_two_to_the_31():
    """Appending to, and attending over, caches of 2.3e9 elements each."""
    b, h, h_kv, d, rows = 17, 8, 8, 128, 131072
    g = torch.Generator(device="cuda").manual_seed(1)
    kc = torch.full((b, h_kv, rows, d), 7.0, dtype=torch.bfloat16, device="cuda")
    vc = torch.full((b, h_kv, rows, d), 7.0, dtype=torch.bfloat16, device="cuda")
    assert kc.numel() > 2 ** 31
    lens = [1] * (b - 2) + [rows - 200, rows]
    for i in (b - 2, b - 1):
        for c in (kc, vc):
            c[i] = torch.randn(h_kv, rows, d, generator=g, device="cuda")
    q, k, v = (torch.randn(b, 1, n, d, generator=g, device="cuda").bfloat16() for n in (h, h_kv, h_kv))
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    at = n - 1
    qn, _, _ = sdpa_qk_norm_rope(q, k, None, None, v=v, kv_rows=at, k_out=kc, v_out=vc)
    assert torch.equal(qn, q.transpose(1, 2))
    for i, r in enumerate(at.tolist()):
        assert torch.equal(kc[i, :, r], k[i, 0]) and torch.equal(vc[i, :, r], v[i, 0])
    assert (kc[:b - 2, :, 1:] == 7).all()  # no other row was touched
    none = torch.empty(h_kv, 0, d, dtype=torch.bfloat16, device="cuda")
    o, lse = sdpa_fwd_prefix(qn, none, none, kc, vc, n)
    torch.cuda.synchronize()
    assert sdpa_device_error() == 0
    assert torch.equal(o[:b - 2, :, 0], v[:b - 2, 0])  # one key: its value
    for i in (b - 2, b - 1):
        for j in range(h):
            m = lens[i]
            close(o[i, j], lse[i, j], attend(qn[i, j], kc[i, j, :m], vc[i, j, :m],
                                             torch.ones(1, m, dtype=torch.bool, device="cuda"), d ** -0.5, 0.0))


@pytest.mark.parametrize("cap", [0.0, 15.0])
@pytest.mark.parametrize("d,d_v", [(64, 64), (128, 128), (192, 128)])
def test_many_new_tokens(d, d_v, cap):
    """A chunk of 300 new tokens of 8 heads a K/V head: 2400 rows in 19 tiles, each
    token seeing the prefix and the own keys up to itself."""
    b, h, h_kv, s_q, s_p, s_max = 2, 8, 1, 300, 150, 700
    g = torch.Generator(device="cuda").manual_seed(d)

    def r(*shape, mul=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * mul).bfloat16()

    q, kp, vp, k, v = (r(b, h, s_q, d, mul=2.0), r(h_kv, s_p, d), r(h_kv, s_p, d_v), r(b, h_kv, s_max, d),
                       r(b, h_kv, s_max, d_v))
    lens = [300, 691]
    o, lse = sdpa_fwd_prefix(q, kp, vp, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), softcap=cap)
    torch.cuda.synchronize()
    assert sdpa_device_error() == 0
    t = torch.arange(s_q, device="cuda")[:, None]
    for i, m in enumerate(lens):
        kk, vv = torch.cat((kp[0], k[i, 0, :m])), torch.cat((vp[0], v[i, 0, :m]))
        seen = torch.arange(s_p + m, device="cuda")[None] <= s_p + m - s_q + t
        for j in range(h):
            close(o[i, j], lse[i, j], attend(q[i, j], kk, vv, seen, d ** -0.5, cap), cap)


@pytest.mark.parametrize("d,d_v", [(64, 64), (128, 128), (192, 128)])
def test_rows_of_no_sequence(d, d_v):
    """Packed rows before the first and behind the last sequence: capped O, LSE, dK and
    dV leave them as they were, dQ leaves them or gives them 0."""
    h, h_kv, total, st = 4, 2, 700, [30, 31, 31, 331, 459, 536]
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v, do = (torch.randn(n, total, w, generator=g, device="cuda").bfloat16()
                   for n, w in ((h, d), (h_kv, d), (h_kv, d_v), (h, d_v)))
    starts = torch.tensor(st, dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(do, 7.0), torch.full((h, total), 7.0, device="cuda")
    pack, kw = (starts, starts, 300, 300), dict(is_causal=True, softcap=20.0)
    sdpa_fwd_varlen(q, k, v, *pack, out=out, lse=lse, **kw)
    no = torch.ones(total, dtype=torch.bool, device="cuda")
    no[st[0]:st[-1]] = False
    assert (out[:, no] == 7).all() and (lse[:, no] == 7).all()
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    for det in (False, True):
        dq, dk, dv = (torch.full_like(x, 7.0) for x in (q, k, v))
        sdpa_bwd_varlen(q, k, v, out, do, lse, *pack, dq=dq, dk=dk, dv=dv, deterministic=det, **kw)
        torch.cuda.synchronize()
        assert (dk[:, no] == 7).all() and (dv[:, no] == 7).all()
        assert (dq[:, no] == (7 if det or d == 192 else 0)).all()
        assert torch.isfinite(dq.float()).all() and not (dq[:, ~no] == 7).all(-1).any()
    assert sdpa_device_error() == 0
