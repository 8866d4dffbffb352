"""Norm, rotation and append into pages (sdpa_qk_norm_rope with kv_slots): the
same bits as into a contiguous cache, in the rows that the slots name and in no other."""
from __future__ import annotations

import pytest
import torch

from scaled_dot_product_06_gb300 import sdpa_qk_norm_rope
from scaled_dot_product_06_gb300.inputs import DTYPES

pytestmark = pytest.mark.gpu

# b, s, h, h_kv, d, d_v, dtype, rot, page, token-major pages
CASES = [
    (1, 1, 1, 1, 64, 64, "bf16", 64, 16, False),
    (5, 1, 8, 2, 128, 128, "bf16", 128, 16, True),
    (3, 77, 6, 3, 192, 128, "fp16", 64, 32, False),
    (1, 500, 4, 4, 64, 64, "fp16", 32, 24, True),      # any page size here
    (64, 1, 32, 4, 128, 128, "bf16", 128, 1, False),
    (2, 300, 40, 8, 128, 64, "bf16", 0, 256, True),
]


def make(c, seed=0):
    b, s, h, h_kv, d, d_v, dt, rot, page, token_major = c
    g = torch.Generator().manual_seed(seed)
    t = DTYPES[dt]

    def r(*shape):
        return torch.randn(*shape, generator=g).to(t).cuda()

    x = {"q": r(b, s, h, d), "k": r(b, s, h_kv, d), "v": r(b, s, h_kv, d_v)}
    kw = {"q_weight": r(d).float(), "k_weight": r(d).float(), "cos": None, "sin": None,
          "positions": torch.randint(0, 900, (b, s), generator=g).to(torch.int32).cuda()}
    if rot:
        ang = torch.rand(900, rot // 2, generator=g) * 6
        kw["cos"], kw["sin"] = ang.cos().cuda(), ang.sin().cuda()
    count = (b * s + page - 1) // page + 3

    def pages(w):
        return r(count, page, h_kv, w).transpose(1, 2) if token_major else r(count, h_kv, page, w)

    slots = torch.randperm(count * page, generator=g)[:b * s].view(b, s).to(torch.int32).cuda()
    return x, kw, pages(d), pages(d_v), slots


def append(x, kw, kp, vp, slots, **more):
    return sdpa_qk_norm_rope(x["q"], x["k"], v=x["v"], kv_slots=slots, k_out=kp, v_out=vp, **kw, **more)


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_rows_named_by_the_slots(c):
    x, kw, kp, vp, slots = make(c)
    page = c[8]
    flat = slots.view(-1)
    # tokens without a slot, and slots that no page has
    for i, bad in zip(range(1, flat.numel(), 7), (-1, kp.shape[0] * page, -(1 << 31), (1 << 31) - 1) * 99):
        flat[i] = bad
    q, k, v = sdpa_qk_norm_rope(x["q"], x["k"], v=x["v"], **kw)
    want_k, want_v = kp.clone(), vp.clone()
    ok = (slots >= 0) & (slots < kp.shape[0] * page)
    at = slots[ok].long()
    want_k[at // page, :, at % page] = k.transpose(1, 2)[ok]
    want_v[at // page, :, at % page] = v.transpose(1, 2)[ok]
    got = append(x, kw, kp, vp, slots)
    assert got[1] is kp and got[2] is vp
    assert torch.equal(got[0], q) and torch.equal(kp, want_k) and torch.equal(vp, want_v)


def test_keys_alone_one_page_and_none():
    x, kw, kp, vp, slots = make((2, 3, 2, 2, 64, 64, "bf16", 32, 16, False))
    one = kp[:1].clone()
    # (a page stride that is none: one page has no second one)
    odd = torch.as_strided(one, one.shape, (3, *one.stride()[1:]))
    s = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    q, k, v = sdpa_qk_norm_rope(x["q"], x["k"], kv_slots=s, k_out=odd, **kw)
    want = sdpa_qk_norm_rope(x["q"], x["k"], **kw)
    assert v is None and torch.equal(q, want[0])
    assert torch.equal(one[0, :, :6], want[1].transpose(0, 1).flatten(1, 2)) and torch.equal(one[0, :, 6:], kp[0, :, 6:])
    none = sdpa_qk_norm_rope(x["q"], x["k"], v=x["v"], kv_slots=s, k_out=kp[:0], v_out=vp[:0], **kw)
    assert torch.equal(none[0], want[0])


def test_the_same_slot_twice_leaves_one_of_the_rows():
    x, kw, kp, vp, slots = make((1, 64, 4, 2, 128, 128, "bf16", 128, 16, False))
    slots[:] = 21
    before = kp.clone()
    append(x, kw, kp, vp, slots)
    rows = sdpa_qk_norm_rope(x["q"], x["k"], **kw)[1]
    for j in range(2):
        assert (kp[1, j, 5] == rows[0, j]).all(-1).any()
    kp[1, :, 5] = before[1, :, 5]
    assert torch.equal(kp, before)


def test_pools_past_32_bits():
    """The last page of a pool of more than 2^31 elements."""
    x, kw, _, _, _ = make((1, 2, 2, 8, 128, 128, "bf16", 128, 64, False))
    count = (1 << 31) // (8 * 64 * 128) + 40
    kp = torch.zeros(count, 8, 64, 128, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    slots = torch.tensor([[count * 64 - 1, (count - 1) * 64]], dtype=torch.int32, device="cuda")
    append(x, kw, kp, vp, slots)
    rows = sdpa_qk_norm_rope(x["q"], x["k"], v=x["v"], **kw)
    for p, r in ((kp, rows[1]), (vp, rows[2])):
        assert torch.equal(p[-1, :, 63], r[0, :, 0]) and torch.equal(p[-1, :, 0], r[0, :, 1])
        assert int(torch.count_nonzero(p[-1, :, 1:63])) == 0 and int(torch.count_nonzero(p[:-1])) == 0


def test_refusals():
    x, kw, kp, vp, slots = make(CASES[1])
    for bad in (dict(kv_slots=slots.long()), dict(kv_slots=slots[:, :0]), dict(kv_slots=slots.cpu()),
                dict(k_out=None), dict(v_out=None), dict(k_out=kp[:, :1]), dict(v_out=vp[:-1]), dict(k_out=kp[0]),
                dict(k_out=kp[:1].expand(kp.shape)), dict(kv_rows=slots[:, 0].contiguous())):
        with pytest.raises(ValueError):
            sdpa_qk_norm_rope(x["q"], x["k"], v=x["v"], **{"kv_slots": slots, "k_out": kp, "v_out": vp, **kw, **bad})
