"""Given outputs, workspaces and keep bits of the wrong size, layout, type or place are
refused on the host by every backward and by the calls around the attention."""
from __future__ import annotations

import pytest
import torch

from scaled_dot_product_06_gb300 import (SDPA_BWD_DKDV, SDPA_BWD_DQ, SDPA_BWD_PREPROCESS, sdpa_bwd, sdpa_bwd_phases,
                                         sdpa_bwd_varlen, sdpa_bwd_workspace_size, sdpa_dropout_mask,
                                         sdpa_fwd, sdpa_fwd_prefix, sdpa_fwd_prefix_workspace_size, sdpa_fwd_varlen,
                                         sdpa_qk_norm_rope_bwd, sdpa_qk_norm_rope_bwd_workspace_size)
from scaled_dot_product_06_gb300.inputs import Shape, make_inputs, make_packed_inputs

pytestmark = pytest.mark.gpu


def u8(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def bad_workspaces(need):
    return (torch.zeros(need, dtype=torch.uint8), u8(1).expand(need), u8(2 * need)[::2], u8((4 * need)).view(4, -1).t())


@pytest.mark.parametrize("softcap", [None, 20.0])
def test_backward(softcap):
    x = make_inputs(Shape(1, 2, 128, 128, 64, 64, 1), "bf16")
    q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "do"))
    kw = dict(is_causal=True, softcap=softcap)
    o, lse = sdpa_fwd(q, k, v, **kw)
    good = sdpa_bwd(q, k, v, o, do, lse, **kw)
    for name, like in (("dq", q), ("dk", k), ("dv", v)):
        wide = torch.empty(*like.shape[:3], 128, dtype=like.dtype, device="cuda")
        for bad in (like[:, :, :64].contiguous(), like.half(), wide[..., :64], like.cpu()):
            with pytest.raises(ValueError, match=name):
                sdpa_bwd(q, k, v, o, do, lse, **{name: bad}, **kw)
    need = sdpa_bwd_workspace_size(1, 2, 128, 128, 64, 64, 1)
    for ws in bad_workspaces(need):
        with pytest.raises(ValueError, match="workspace"):
            sdpa_bwd(q, k, v, o, do, lse, workspace=ws, **kw)
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        sdpa_bwd(q, k, v, o, do, lse, workspace=u8(512), **kw)  # less than the row statistics
    # a workspace of another type counts by its bytes
    fp = torch.empty((need + 3) // 4, device="cuda")
    again = sdpa_bwd(q, k, v, o, do, lse, workspace=fp, **kw)
    assert torch.equal(again[1], good[1]) and torch.equal(again[2], good[2])


@pytest.mark.parametrize("softcap", [None, 20.0])
def test_keep_bits(softcap):
    x = make_inputs(Shape(1, 2, 128, 128, 64, 64), "bf16")
    q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "do"))
    kw = dict(softcap=softcap, dropout_p=0.5, seed=1, offset=0)
    mask = sdpa_dropout_mask(1, 2, 128, 128, 0.5, 1, 0)
    o, lse = sdpa_fwd(q, k, v, dropout_mask=mask, **kw)
    for bad in (mask[:-1], mask.cpu(), mask.long(), torch.cat((mask, mask))[::2]):
        with pytest.raises(ValueError, match="dropout_mask"):
            sdpa_fwd(q, k, v, dropout_mask=bad, **kw)
        with pytest.raises(ValueError, match="dropout_mask"):
            sdpa_bwd(q, k, v, o, do, lse, dropout_mask=bad, **kw)
    p = make_packed_inputs(2, 100, 100, 64, 64, "bf16")
    pq, pk, pv = (p[n].cuda() for n in ("q", "k", "v"))
    st = torch.tensor([0, 40, 100], dtype=torch.int32, device="cuda")
    small = sdpa_dropout_mask(2, 2, 40, 40, 0.5, 1, 0)  # the frame is of the longest: 60
    with pytest.raises(ValueError, match="dropout_mask"):
        sdpa_fwd_varlen(pq, pk, pv, st, st, 60, 60, dropout_mask=small, **kw)
    with pytest.raises(ValueError, match="out"):
        sdpa_dropout_mask(1, 2, 128, 128, 0.5, 1, 0, out=torch.empty(4 * mask.numel(), dtype=torch.int32,
                                                                    device="cuda")[::2])


def test_packed_backward():
    p = make_packed_inputs(2, 100, 100, 64, 64, "bf16")
    q, k, v, do = (p[n].cuda() for n in ("q", "k", "v", "do"))
    st = torch.tensor([0, 40, 100], dtype=torch.int32, device="cuda")
    o, lse = sdpa_fwd_varlen(q, k, v, st, st, 60, 60)
    for name, bad in (("dq", q[:, :90]), ("dk", k.float()), ("dv", v.transpose(0, 1).contiguous())):
        with pytest.raises(ValueError, match=name):
            sdpa_bwd_varlen(q, k, v, o, do, lse, st, st, 60, 60, **{name: bad})
    for ws in bad_workspaces(1 << 20):
        with pytest.raises(ValueError, match="workspace"):
            sdpa_bwd_varlen(q, k, v, o, do, lse, st, st, 60, 60, workspace=ws)


def test_around_the_attention():
    g = torch.Generator(device="cuda").manual_seed(0)

    def r(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    args = (r(2, 4, 1, 64), r(2, 300, 64), r(2, 300, 64), r(2, 2, 16, 64), r(2, 2, 16, 64),
            torch.tensor([3, 16], dtype=torch.int32, device="cuda"))
    need = sdpa_fwd_prefix_workspace_size(2, 4, 2, 1, 300, 16, 64, 64)
    for ws in bad_workspaces(need):
        with pytest.raises(ValueError, match="workspace"):
            sdpa_fwd_prefix(*args, workspace=ws)
    x, dy, w = r(1, 8, 2, 64), r(1, 2, 8, 64), torch.ones(64, device="cuda")
    need = sdpa_qk_norm_rope_bwd_workspace_size(1, 8, 2, 2, 64, 64)
    for ws in bad_workspaces(need):
        with pytest.raises(ValueError, match="workspace"):
            sdpa_qk_norm_rope_bwd(dy, dy, x, x, None, None, q_weight=w, k_weight=w, workspace=ws)


@pytest.mark.parametrize("deterministic", [False, True])
def test_phases_with_stand_ins(deterministic):
    """A phase takes stand-ins for the gradients that it does not write."""
    x = make_inputs(Shape(1, 2, 128, 256, 64, 64), "bf16")
    q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "do"))
    kw = dict(is_causal=True, softcap=20.0, deterministic=deterministic)
    o, lse = sdpa_fwd(q, k, v, is_causal=True, softcap=20.0)
    want = sdpa_bwd(q, k, v, o, do, lse, **kw)
    ws = u8(sdpa_bwd_workspace_size(1, 2, 128, 256, 64, 64, 2, deterministic))
    one = torch.empty(64, dtype=torch.bfloat16, device="cuda")
    dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
    call = dict(workspace=ws, **kw)
    sdpa_bwd_phases(SDPA_BWD_PREPROCESS, q, k, v, o, do, lse, dq=one, dk=one, dv=one, **call)
    sdpa_bwd_phases(SDPA_BWD_DKDV, q, k, v, o, do, lse, dq=dq, dk=dk, dv=dv, **call)
    sdpa_bwd_phases(SDPA_BWD_DQ, q, k, v, o, do, lse, dq=dq, dk=dk, dv=dv, **call)
    torch.cuda.synchronize()
    assert torch.equal(dk, want[1]) and torch.equal(dv, want[2])
    if deterministic:
        assert torch.equal(dq, want[0])
    for phase, kws in ((SDPA_BWD_DKDV, dict(dq=dq, dk=one, dv=dv)), (SDPA_BWD_DQ, dict(dq=one, dk=dk, dv=dv))):
        with pytest.raises(ValueError):
            sdpa_bwd_phases(phase, q, k, v, o, do, lse, **kws, **call)
