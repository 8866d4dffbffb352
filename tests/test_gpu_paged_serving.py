"""The paged cache's operators as a server uses them together: prompts packed
into pages, decoding steps in one captured graph, requests that end and begin."""
from __future__ import annotations

import math

import pytest
import torch

from capped_bounds import u_of
from scaled_dot_product_06_gb300 import (sdpa_device_error, sdpa_fwd_paged, sdpa_fwd_varlen, sdpa_page_slots,
                                         sdpa_qk_norm_rope)

pytestmark = pytest.mark.gpu

B, H, H_KV, D, PAGE, POOL, WIDE = 6, 8, 2, 64, 16, 60, 12
STEPS = 40


def test_serving_loop_equals_the_whole_sequences():
    """Every token's attention in the loop, step by step over pages, against one plain
    fp64 attention over its sequence's rows as the norm and rotation leave them."""
    dt = torch.bfloat16
    g = torch.Generator().manual_seed(1)
    ang = torch.rand(200, D // 2, generator=g) * 6
    cos, sin = ang.cos().cuda(), ang.sin().cuda()
    wq, wk = (1 + 0.1 * torch.randn(2, D, generator=g)).cuda()
    kp = torch.full((POOL, H_KV, PAGE, D), float("nan"), dtype=dt, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    table = torch.full((B, WIDE), -1, dtype=torch.int32, device="cuda")
    ring = torch.randperm(POOL, generator=g).to(torch.int32).cuda()
    span = torch.tensor([0, POOL], dtype=torch.int64, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    kw = dict(q_weight=wq, k_weight=wk)

    def randn(*shape):
        return torch.randn(*shape, generator=g).to(dt).cuda()

    # what each request's sequence has seen: rows of k and v as the attention takes them
    rows = [[torch.zeros(H_KV, 0, D, dtype=dt, device="cuda")] * 2 for _ in range(B)]

    def keep(i, k, v):
        rows[i] = [torch.cat((rows[i][0], k), 1), torch.cat((rows[i][1], v), 1)]

    def compare(q, i, got):  # q [H, t, D]: the newest t tokens of request i
        k, v = (x.double().repeat_interleave(H // H_KV, 0) for x in rows[i])
        s = q.double() @ k.transpose(1, 2) / math.sqrt(D)
        n, t = k.shape[1], q.shape[1]
        at = torch.arange(n, device="cuda")
        s = s.masked_fill(at > (n - t + torch.arange(t, device="cuda"))[:, None], float("-inf"))
        p = torch.softmax(s, -1)
        # P and O rounded once, scores and sums in fp32
        lim = (u_of(dt) + 2.0 ** -10) * (p @ v.abs()) + u_of(dt) * (p @ v).abs()
        assert ((got.double() - p @ v).abs() <= lim).all()

    # ---- prompts, packed
    prompts = [33, 0, 1, 100, 16, 70]
    total = 256  # entries; the tail is padding
    new.copy_(torch.tensor(prompts, dtype=torch.int32))
    slots, positions, starts, *_ = sdpa_page_slots(lens, new, table, ring, span, PAGE, rows=total, seqlens_out=lens,
                                                   free_range_out=span)
    q, k, v = randn(1, total, H, D), randn(1, total, H_KV, D), randn(1, total, H_KV, D)
    args = dict(positions=positions[None], **kw)
    q1, _, _ = sdpa_qk_norm_rope(q, k, cos, sin, v=v, kv_slots=slots[None], k_out=kp, v_out=vp, **args)
    _, k1, v1 = sdpa_qk_norm_rope(q, k, cos, sin, v=v, **args)
    o, _ = sdpa_fwd_varlen(q1[0], k1[0], v1[0], starts, starts, max(prompts), max(prompts), is_causal=True)
    assert starts.tolist() == [0, 33, 33, 34, 134, 150, 220] and lens.tolist() == prompts
    first = starts.tolist()
    for i, n in enumerate(prompts):
        sl = slice(first[i], first[i] + n)
        keep(i, k1[0, :, sl], v1[0, :, sl])
        if n:
            compare(q1[0, :, sl], i, o[:, sl])
            # the last 16 of them once more, over the pages
            t = min(n, 16)
            one = sdpa_fwd_paged(q1[0, :, first[i] + n - t:first[i] + n][None].contiguous(), kp, vp, table[i:i + 1],
                                 lens[i:i + 1])
            compare(q1[0, :, first[i] + n - t:first[i] + n], i, one[0][0])

    # ---- decoding: one token a request, captured once
    q, k, v = (torch.zeros(B, 1, n, D, dtype=dt, device="cuda") for n in (H, H_KV, H_KV))

    def step():
        slots, positions, _, _, _ = sdpa_page_slots(lens, new, table, ring, span, PAGE, width=1, seqlens_out=lens,
                                                    free_range_out=span)
        q1, _, _ = sdpa_qk_norm_rope(q, k, cos, sin, v=v, positions=positions, kv_slots=slots, k_out=kp, v_out=vp, **kw)
        o, lse = sdpa_fwd_paged(q1, kp, vp, table, lens)
        return q1, positions, o, lse

    new.fill_(0)
    step()  # (idle: nothing is stored)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q1, positions, o, lse = step()
    length = list(prompts)
    for n in range(STEPS):
        active = [1] * B
        if n % 9 == 4:
            active[n % B] = -1  # ends; its row is another request's in the next step
        if n % 5 == 2:
            active[(n + 3) % B] = 0
        new.copy_(torch.tensor(active, dtype=torch.int32))
        q.copy_(randn(B, 1, H, D))
        k.copy_(randn(B, 1, H_KV, D))
        v.copy_(randn(B, 1, H_KV, D))
        graph.replay()
        torch.cuda.synchronize()
        assert sdpa_device_error() == 0
        plain_k = sdpa_qk_norm_rope(q, k, cos, sin, positions=positions, **kw)[1]
        for i, a in enumerate(active):
            if a < 0:
                rows[i] = [x[:, :0] for x in rows[i]]
                length[i] = 0
            elif a and length[i] < WIDE * PAGE:
                assert int(positions[i, 0]) == length[i]
                keep(i, plain_k[i], v[i].transpose(0, 1))
                length[i] += 1
                compare(q1[i], i, o[i])
        assert lens.tolist() == length
    # every page is owned once or free
    owned = [int(x) for i in range(B) for x in table[i, :-(-length[i] // PAGE)].tolist()]
    head, tail = span.tolist()
    owned += [int(ring[j % POOL]) for j in range(head, tail)]
    assert sorted(owned) == list(range(POOL))


def test_captured_on_streams_that_fork_and_join():
    """Slots on one stream, the queries' copy on another, norm and attention behind both;
    replays equal the calls one by one."""
    dt, b, h, h_kv, d, page, pool = torch.float16, 5, 8, 2, 64, 16, 400
    g = torch.Generator().manual_seed(2)

    def randn(*shape):
        return torch.randn(*shape, generator=g).to(dt).cuda()

    q0, k, v = randn(b, 1, h, d), randn(b, 1, h_kv, d), randn(b, 1, h_kv, d)
    ang = torch.rand(2000, d // 2, generator=g).cuda()
    cos, sin = ang.cos(), ang.sin()
    pages = [randn(pool, h_kv, page, d) for _ in range(2)]
    ring = torch.randperm(pool, generator=g).to(torch.int32).cuda()
    new = torch.tensor([1, 1, 0, 1, 1], dtype=torch.int32).cuda()
    first = torch.tensor([900, 0, 33, 15, 640], dtype=torch.int32).cuda()

    def state():
        table = torch.full((b, 64), -1, dtype=torch.int32, device="cuda")
        used = 0
        for i, n in enumerate(first.tolist()):
            own = -(-n // page)
            table[i, :own] = ring[used:used + own]
            used += own
        span = torch.tensor([used, pool], dtype=torch.int64, device="cuda")
        return dict(table=table, ring=ring.clone(), span=span, lens=first.clone(), q=torch.zeros_like(q0),
                    kp=pages[0].clone(), vp=pages[1].clone())

    def slots_of(s):
        return sdpa_page_slots(s["lens"], new, s["table"], s["ring"], s["span"], page, width=1, seqlens_out=s["lens"],
                               free_range_out=s["span"])[:2]

    def attend(s, slots, positions):
        q1, _, _ = sdpa_qk_norm_rope(s["q"], k, cos, sin, v=v, positions=positions, kv_slots=slots, k_out=s["kp"],
                                     v_out=s["vp"])
        return sdpa_fwd_paged(q1, s["kp"], s["vp"], s["table"], s["lens"])

    a, e = state(), state()
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for s in side:
            s.wait_stream(main)
        with torch.cuda.stream(side[0]):
            slots, positions = slots_of(a)
        with torch.cuda.stream(side[1]):
            a["q"].copy_(q0)
        for s in side:
            main.wait_stream(s)
        got = attend(a, slots, positions)
    for _ in range(20):
        graph.replay()
        e["q"].copy_(q0)
        want = attend(e, *slots_of(e))
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert all(torch.equal(a[n], e[n]) for n in a)
