"""Attention over a paged cache (sdpa_fwd_paged) against plain fp64 arithmetic,
element by element; bounds in paged_ref."""
from __future__ import annotations

import concurrent.futures
import math

import pytest
import torch

from paged_ref import check, make
from scaled_dot_product_06_gb300 import (sdpa_device_error, sdpa_fwd_paged, sdpa_fwd_paged_workspace_size,
                                         sdpa_fwd_prefix)
from scaled_dot_product_06_gb300.inputs import DTYPES

pytestmark = pytest.mark.gpu

NAN = float("nan")


def cuda(x):
    return {n: t.cuda() for n, t in x.items()}


def call(x, **kw):
    return sdpa_fwd_paged(**cuda(x), **kw)


# (b, h, h_kv, s_q, lens, page, d, d_v, dtype, cap, left, token-major)
CASES = [
    (1, 1, 1, 1, [1], 8, 64, 64, "bf16", 0.0, -1, False),
    (2, 8, 1, 1, [1, 17], 16, 64, 64, "fp16", 0.0, -1, False),
    (4, 8, 2, 1, [128, 129, 127, 256], 16, 128, 128, "bf16", 0.0, -1, True),
    (3, 6, 3, 1, [200, 0, 333], 32, 192, 128, "fp16", 30.0, -1, False),       # a sequence without a key
    (3, 4, 4, 1, [0, 0, 0], 16, 128, 128, "bf16", 0.0, -1, False),            # all of them
    (2, 4, 2, 4, [4, 300], 64, 128, 128, "bf16", 0.0, -1, False),             # drafted tokens
    (3, 4, 2, 5, [3, 0, 131], 16, 64, 64, "bf16", 20.0, -1, True),            # fewer keys than tokens
    (2, 16, 1, 1, [700, 45], 8, 128, 128, "fp16", 0.0, -1, False),            # R = 16, the smallest pages
    (2, 17, 1, 1, [700, 45], 128, 128, 128, "bf16", 0.0, -1, False),          # R = 17
    (2, 32, 1, 1, [260, 1025], 256, 64, 64, "bf16", 50.0, -1, True),          # R = 32
    (2, 11, 1, 3, [260, 1025], 1024, 128, 128, "bf16", 0.0, -1, False),       # R = 33: both warpgroups
    (2, 64, 1, 1, [513, 90], 16, 192, 128, "bf16", 0.0, -1, False),           # R = 64
    (2, 64, 1, 1, [513, 90], 32, 64, 64, "fp16", 15.0, -1, False),
    (1, 65, 1, 1, [400], 16, 128, 128, "bf16", 0.0, -1, False),               # R = 65: two row blocks
    (2, 16, 2, 20, [20, 500], 64, 64, 64, "bf16", 0.0, -1, True),             # R = 160: three
    (1, 8, 8, 1, [20000], 64, 64, 64, "bf16", 0.0, -1, False),                # cut many times
    (1, 16, 1, 1, [33333], 16, 128, 128, "bf16", 0.0, -1, False),             # by every CTA
    (3, 4, 1, 1, [9000, 1, 4097], 128, 192, 128, "fp16", 0.0, -1, True),
    (200, 4, 1, 1, [(37 * i) % 300 for i in range(200)], 16, 64, 64, "bf16", 0.0, -1, False),  # many units a CTA
    (400, 2, 1, 1, [i % 3 for i in range(400)], 16, 128, 128, "fp16", 0.0, -1, False),  # more than threads
    (2, 8, 2, 1, [900, 77], 16, 128, 128, "bf16", 0.0, 100, False),           # windows
    (2, 8, 2, 1, [900, 77], 64, 64, 64, "bf16", 0.0, 0, True),                # a token sees itself
    (3, 8, 2, 3, [1000, 130, 2], 32, 128, 128, "fp16", 25.0, 127, False),
    (2, 40, 1, 2, [3001, 640], 128, 192, 128, "bf16", 0.0, 1000, False),
    (2, 4, 2, 6, [300, 5], 16, 64, 64, "bf16", 0.0, 2, False),
    # many units, one of them in so many parts that they are joined in groups
    (90, 4, 1, 1, [1] * 45 + [40000] + [3] * 44, 16, 128, 128, "bf16", 0.0, -1, False),
    (80, 40, 1, 1, [130] * 79 + [30000], 64, 64, 64, "fp16", 0.0, -1, True),    # by halves of the rows
    (80, 16, 1, 1, [20000] + [0, 300] * 39 + [5000], 128, 192, 128, "bf16", 0.0, -1, False),
    (100, 2, 1, 2, [(i * 331) % 2500 for i in range(100)], 32, 128, 128, "bf16", 30.0, 900, False),
]


def case_id(c):
    return f"b{c[0]}h{c[1]}kv{c[2]}q{c[3]}-n{max(c[4])}-p{c[5]}-d{c[6]}-{c[8]}-cap{c[9]}-w{c[10]}"


def inputs(c, **kw):
    return make(c[0], c[1], c[2], c[3], c[4], c[5], c[6], c[7], DTYPES[c[8]], seed=len(c[4]) + c[5],
                token_major=c[11], **kw)


@pytest.mark.parametrize("c", CASES, ids=case_id)
def test_matches_reference(c):
    x = inputs(c)
    kw = dict(softcap=c[9], window_left=c[10])
    got = call(x, **kw)
    check(x, got, 1 / math.sqrt(c[6]), c[9], c[10])
    again = call(x, **kw)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("scale", [-0.2, 0.0, 0.3])
@pytest.mark.parametrize("cap", [0.0, 7.0])
def test_scales(scale, cap):
    x = make(2, 4, 2, 2, [139, 2], 16, 64, 64, torch.bfloat16)
    check(x, call(x, scale=scale, softcap=cap), scale, cap)


def test_scores_far_apart():
    """A running maximum that jumps between tiles and parts, and far below what
    another warp's keys have."""
    for mul, n in ((40.0, [900, 300]), (6.0, [5000, 45])):
        x = make(2, 8, 2, 1, n, 16, 128, 128, torch.bfloat16, q_mul=mul)
        ids = x["block_table"][0]
        for j, f in ((5, 3), (500, 8), (130, 2), (899, 12)):
            x["k_pages"][ids[j // 16], :, j % 16] *= f
        check(x, call(x), 1 / math.sqrt(128))
        check(x, call(x, softcap=20.0), 1 / math.sqrt(128), 20.0)


def test_what_lies_elsewhere_under_load():
    """Every SM streaming, ragged lengths, a window: what no token sees changes no bit."""
    lens = [(i * 991) % 3000 + 1 for i in range(64)]
    for d, d_v in ((64, 64), (128, 128), (192, 128)):
        x = make(64, 8, 4, 1, lens, 32, d, d_v, torch.bfloat16, q_mul=1.0)
        y = dict(x, k_pages=x["k_pages"].nan_to_num(0.0, 0.0, 0.0), v_pages=x["v_pages"].nan_to_num(0.0, 0.0, 0.0))
        y["block_table"] = torch.where(x["block_table"] < 0, 0, x["block_table"])
        gx, gy = cuda(x), cuda(y)
        for left in (-1, 700):
            want = sdpa_fwd_paged(**gy, window_left=left)
            assert torch.isfinite(want[0]).all()
            for _ in range(5):
                got = sdpa_fwd_paged(**gx, window_left=left)
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert sdpa_device_error() == 0


def test_pages_before_the_window_are_not_read():
    """A window's pages alone: those before it have been given away."""
    x = make(2, 8, 2, 1, [1000, 400], 16, 128, 128, torch.bfloat16)
    full = call(x, window_left=200)
    y = dict(x, block_table=x["block_table"].clone(), k_pages=x["k_pages"].clone(), v_pages=x["v_pages"].clone())
    for i, n in enumerate((1000, 400)):
        for c in range((n - 201) // 16):
            pg = int(x["block_table"][i, c])
            y["k_pages"][pg], y["v_pages"][pg], y["block_table"][i, c] = NAN, NAN, -1
    got = call(y, window_left=200)
    assert torch.equal(got[0], full[0]) and torch.equal(got[1], full[1])


def test_page_numbers_outside_the_pool_read_as_zeros():
    x = make(2, 4, 2, 1, [100, 64], 16, 64, 64, torch.bfloat16)
    y = dict(x, block_table=x["block_table"].clone())
    ids = [int(x["block_table"][0, c]) for c in (1, 4)]
    z = dict(x, k_pages=x["k_pages"].clone(), v_pages=x["v_pages"].clone())
    for pg in ids:
        z["k_pages"][pg], z["v_pages"][pg] = 0.0, 0.0
    want = call(z)
    for bad in (-1, x["k_pages"].shape[0], 1 << 30, -(1 << 31)):
        y["block_table"][0, 1] = y["block_table"][0, 4] = bad
        got = call(y)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_lengths_past_the_table():
    x = make(2, 4, 2, 1, [64, 40], 16, 64, 64, torch.bfloat16)
    x["block_table"] = x["block_table"][:, :4].contiguous()
    y = dict(x, seqlens_k=torch.tensor([1 << 30, -3], dtype=torch.int32))
    got = call(y)
    want = call(x)
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[1][0], want[1][0])
    assert (got[0][1] == 0).all() and torch.isneginf(got[1][1]).all()
    # no pages, no table
    for z in (dict(y, k_pages=x["k_pages"][:0], v_pages=x["v_pages"][:0]), dict(y, block_table=x["block_table"][:, :0])):
        got = call(z)
        assert (got[0] == 0).all() and torch.isneginf(got[1]).all()
    for z in (dict(x, q=x["q"][:, :, :0]), dict(x, q=x["q"][:0], block_table=x["block_table"][:0],
                                                seqlens_k=x["seqlens_k"][:0])):
        got = call(z)
        assert got[0].numel() == 0 and got[1].numel() == 0


def test_values_that_are_not_a_number():
    """A key or query that is none reaches exactly the rows that see it."""
    for c in (CASES[5], CASES[2], CASES[11], CASES[15]):
        x = inputs(c)
        b, h, h_kv, s_q, lens, page = c[:6]
        group = h // h_kv
        clean = call(x)
        n = lens[-1]
        for j in sorted({0, n // 2, n - 1}):
            y = dict(x, k_pages=x["k_pages"].clone())
            y["k_pages"][int(x["block_table"][b - 1, j // page]), 0, j % page, 3] = NAN
            hit = torch.zeros(b, h, s_q, dtype=torch.bool)
            for t in range(s_q):
                hit[b - 1, :group, t] = j <= n - s_q + t
            expect(call(y), clean, hit.cuda())
        y = dict(x, q=x["q"].clone())
        y["q"][b - 1, h - 1, s_q - 1, 0] = NAN
        hit = torch.zeros(b, h, s_q, dtype=torch.bool)
        hit[b - 1, h - 1, s_q - 1] = True
        expect(call(y), clean, hit.cuda())
        expect(call(y, softcap=30.0), call(x, softcap=30.0), hit.cuda())


def expect(got, clean, hit):
    assert torch.isnan(got[0][hit]).all() and torch.isnan(got[1][hit]).all()
    assert torch.equal(got[0][~hit], clean[0][~hit]) and torch.equal(got[1][~hit], clean[1][~hit])


@pytest.mark.parametrize("scale", [0.1, -0.1])
def test_infinite_scores(scale):
    """A key that is infinite in one element: rows with a score of +inf are NaN, rows
    with -inf give it no weight."""
    x = make(2, 8, 2, 1, [300, 77], 16, 64, 64, torch.bfloat16)
    clean = call(x, scale=scale)
    y = dict(x, k_pages=x["k_pages"].clone())
    y["k_pages"][int(x["block_table"][0, 8]), 0, 3, 7] = float("inf")
    o, lse = call(y, scale=scale)
    up = (x["q"][:, :, :, 7].float() * scale > 0).cuda()
    up[:, 4:] = False
    up[1:] = False
    assert torch.isnan(o[up]).all() and torch.isnan(lse[up]).all()
    assert torch.isfinite(o[~up].float()).all() and torch.isfinite(lse[~up]).all()
    assert torch.equal(o[:, 4:], clean[0][:, 4:]) and torch.equal(o[1], clean[0][1])


def test_writes_stay_inside():
    x = make(3, 6, 2, 2, [2, 950, 77], 16, 128, 128, torch.bfloat16)
    need = sdpa_fwd_paged_workspace_size(6, 2, 2, 128, 128, 16, 60)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    buf = torch.full((3 * 6 * 2 * 128 + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    lb = torch.full((3 * 6 * 2 + 8,), 7.0, device="cuda")
    wide = torch.full((3, 80), 1 << 30, dtype=torch.int32, device="cuda")
    w = x["block_table"].shape[1]
    wide[:, 5:5 + w] = x["block_table"].cuda()
    g = cuda(x)
    g["block_table"] = wide[:, 5:5 + w]
    before = {n: t.clone() for n, t in g.items()}
    out, lse = buf[64:-64].view(3, 6, 2, 128), lb[4:-4].view(3, 6, 2)
    got = sdpa_fwd_paged(**g, out=out, lse=lse, workspace=ws[256:256 + need])
    assert got[0] is out and got[1] is lse
    check(x, got, 1 / math.sqrt(128))
    assert (ws[:256] == 0x5A).all() and (ws[256 + need:] == 0x5A).all()
    assert (buf[:64] == 7).all() and (buf[-64:] == 7).all() and (lb[:4] == 7).all() and (lb[-4:] == 7).all()
    for n, t in g.items():
        assert torch.equal(t.view(torch.int16) if t.dtype == torch.bfloat16 else t,
                           before[n].view(torch.int16) if t.dtype == torch.bfloat16 else before[n]), n


def test_pools_past_32_bits():
    """Sequences in the last pages of pools of more than 2^31 elements."""
    x = make(2, 8, 8, 1, [200, 130], 64, 128, 128, torch.bfloat16, garbage=False)
    want = call(x)
    count, extra = x["k_pages"].shape[0], (1 << 31) // (8 * 64 * 128) + 11
    g = cuda(x)
    for n in ("k_pages", "v_pages"):
        big = torch.full((extra + count, 8, 64, 128), NAN, dtype=torch.bfloat16, device="cuda")
        big[extra:] = g[n]
        g[n] = big
    g["block_table"] = torch.where(g["block_table"] >= 0, g["block_table"] + extra, -1).to(torch.int32)
    got = sdpa_fwd_paged(**g)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("batches,more", [((3, 1), 0), ((80, 50), 0), ((80, 50), 700)],
                         ids=["many parts", "whole", "few parts"])
def test_captured_graphs_that_share_a_workspace(batches, more):
    """Two captured calls with one workspace, replayed in turn on lengths that change,
    and that a copy within the graph brings."""
    page, h_kv = 16, 2
    lens = [6000 // b + 600 + more for b in batches]
    xs = [make(b, 16, h_kv, 1, [n] * b, page, 128, 128, torch.bfloat16, seed=b, garbage=False)
          for b, n in zip(batches, lens)]
    ws = torch.full((max(sdpa_fwd_paged_workspace_size(16, h_kv, 1, 128, 128, page, x["block_table"].shape[1])
                         for x in xs),), 0xFF, dtype=torch.uint8, device="cuda")
    gs = [cuda(x) for x in xs]
    news = [g["seqlens_k"].clone() for g in gs]
    graphs, outs = [], []
    for g, new in zip(gs, news):
        sdpa_fwd_paged(**g, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g["seqlens_k"].copy_(new)
            outs.append(sdpa_fwd_paged(**g, workspace=ws))
        graphs.append(graph)
    rng = torch.Generator().manual_seed(3)
    for step in range(8):
        for g, new, graph, out, n in zip(gs, news, graphs, outs, lens):
            new.copy_(torch.randint(0, n + 1, new.shape, generator=rng).to(torch.int32))
            graph.replay()
            if step % 2:
                graph.replay()
            want = sdpa_fwd_paged(**g)
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
            if step % 3 == 0:
                ws.random_(0, 256)
    assert sdpa_device_error() == 0


@pytest.mark.parametrize("c", [CASES[15], CASES[25], CASES[26], CASES[28]], ids=case_id)
def test_workspaces_of_any_contents(c):
    """What the workspace holds, another call's leftovers or anything, changes no bit."""
    x = cuda(inputs(c, garbage=False))
    kw = dict(softcap=c[9], window_left=c[10])
    want = sdpa_fwd_paged(**x, **kw)
    need = sdpa_fwd_paged_workspace_size(c[1], c[2], c[3], c[6], c[7], c[5], x["block_table"].shape[1])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for fill in (0, 0xFF, 0x80, None, None):
        if fill is not None:
            ws.fill_(fill)
        got = sdpa_fwd_paged(**x, **kw, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_streams_at_once():
    x = [cuda(make(8, 8, 2, 1, [4000 - 400 * i for i in range(8)], 16, 128, 128, torch.bfloat16, seed=s))
         for s in range(2)]
    want = [sdpa_fwd_paged(**g) for g in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    for _ in range(20):
        got = [sdpa_fwd_paged(**g, stream=s) for g, s in zip(x, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("long", [448, 1200], ids=["whole", "cut"])
@pytest.mark.parametrize("h,d,d_v,t", [(3, 64, 64, "bf16"), (12, 128, 128, "fp16"), (48, 128, 128, "bf16"),
                                       (6, 192, 128, "bf16"), (36, 192, 128, "fp16")])
def test_short_units_one_behind_another(h, d, d_v, t, long):
    """More units a CTA than buffers of queries, of none to a few tiles in all orders."""
    lens = [(0, 1, 130, 257, 16, 128, 129, 384)[(i * i + 3 * i) % 8] for i in range(160)]
    lens[77] = long
    x = make(160, h, 3, 1, lens, 32, d, d_v, DTYPES[t], seed=d + h)
    check(x, call(x), 1 / math.sqrt(d))


@pytest.mark.parametrize("left,count", [(40, 8), (383, 8), (384, 8), (385, 8), (383, 128), (894, 128), (895, 128),
                                        (896, 128)], ids=lambda n: str(n))
def test_windows_of_a_few_tiles(left, count):
    """Windows around the four and eight tiles up to which few and many units stay whole, at
    all places of a tile."""
    lens = [1300 + i * 128 // count + i for i in range(count)] + [0, 1, 384, 385, 386]
    x = make(len(lens), 4, 2, 2, lens, 32, 64, 64, torch.bfloat16, seed=left)
    check(x, call(x, window_left=left), 1 / 8, left=left)


@pytest.mark.parametrize("count", [1, 18, 19, 75, 76, 77, 200])
@pytest.mark.parametrize("longest", [480, 992, 1000])
def test_units_cut_or_whole(count, longest):
    """Ragged sequences on both sides of the sizes and counts at which units are cut."""
    lens = [(longest * (7 * i + 3)) // 11 % longest for i in range(count - 1)] + [longest]
    x = make(count, 2, 2, 1, lens, 16, 64, 64, torch.float16, seed=count)
    check(x, call(x), 1 / 8)


def test_captured_calls_that_allocate():
    """Captured calls without a given workspace: each one's is handed on within the graph."""
    lens = [700, 3000, 1, 640, 2048, 999]
    xs = [cuda(make(6, 8, 2, 1, lens, 16, 64, 64, torch.float16, seed=s, garbage=False)) for s in range(2)]
    need = sdpa_fwd_paged_workspace_size(8, 2, 1, 64, 64, 16, xs[0]["block_table"].shape[1])
    assert need > 0
    sdpa_fwd_paged(**xs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = []
        for x in xs:
            outs.append(sdpa_fwd_paged(**x))
            torch.empty(need, dtype=torch.uint8, device="cuda").fill_(0xA5)
    for step in range(6):
        for x in xs:
            x["seqlens_k"].copy_(torch.tensor([max(n - 37 * step, 0) for n in lens], dtype=torch.int32))
        graph.replay()
        for x, out in zip(xs, outs):
            want = sdpa_fwd_paged(**x)
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_two_threads_at_once():
    x = [cuda(make(8, 8, 2, 1, [4000 - 400 * i for i in range(8)], 16, 128, 128, torch.bfloat16, seed=s))
         for s in range(2)]
    want = [sdpa_fwd_paged(**g) for g in x]
    torch.cuda.synchronize()

    def calls(i):
        stream = torch.cuda.Stream()
        return all(torch.equal(a, b) for _ in range(40) for a, b in zip(finished(i, stream), want[i]))

    def finished(i, stream):
        got = sdpa_fwd_paged(**x[i], stream=stream)
        stream.synchronize()
        return got

    with concurrent.futures.ThreadPoolExecutor(2) as pool:
        assert all(pool.map(calls, range(2)))


def test_equals_the_contiguous_cache():
    """The same keys in a contiguous cache: the other operator's result within both
    roundings of O."""
    lens = [900, 1, 333, 512]
    x = make(4, 16, 4, 1, lens, 16, 128, 128, torch.bfloat16)
    k, v = torch.zeros(4, 4, 900, 128).bfloat16(), torch.zeros(4, 4, 900, 128).bfloat16()
    for i, n in enumerate(lens):
        for name, c in (("k_pages", k), ("v_pages", v)):
            ids = x["block_table"][i, :(n + 15) // 16].long()
            c[i, :, :n] = x[name][ids].transpose(0, 1).flatten(1, 2)[:, :n]
    e = torch.zeros(4, 0, 128).bfloat16().cuda()
    o, lse = sdpa_fwd_prefix(x["q"].cuda(), e, e, k.cuda(), v.cuda(), x["seqlens_k"].cuda())
    got = call(x)
    assert (got[1] - lse).abs().max() <= 2.0 ** -17 * (1 + lse.abs().max())
    check(x, (o, lse), 1 / math.sqrt(128))


def test_refusals():
    x = cuda(make(2, 4, 2, 1, [30, 40], 16, 64, 64, torch.bfloat16))
    sdpa_fwd_paged(**x)
    t = x["block_table"]
    for bad in (dict(q=x["q"].float()), dict(q=x["q"].half()), dict(k_pages=x["k_pages"][:, :1]),
                dict(v_pages=x["v_pages"][:-1]), dict(k_pages=x["k_pages"][..., :32]), dict(block_table=t.long()),
                dict(block_table=t[:1]), dict(block_table=t[:, ::2]), dict(block_table=t[:1].expand(t.shape)),
                dict(seqlens_k=x["seqlens_k"].long()), dict(seqlens_k=x["seqlens_k"].cpu()),
                dict(out=torch.empty(2, 4, 1, 128, dtype=torch.bfloat16, device="cuda")),
                dict(lse=torch.empty(2, 4, 1, dtype=torch.bfloat16, device="cuda")),
                dict(q=x["q"].expand(2, 4, 1, 64)[:, ::2]), dict(workspace=torch.empty(4, 9, device="cuda").t())):
        with pytest.raises(ValueError):
            sdpa_fwd_paged(**{**x, **bad})
    odd = torch.zeros(9, 2, 12, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(k_pages=odd, v_pages=odd), dict(k_pages=x["k_pages"][:1].expand(x["k_pages"].shape)), dict(softcap=-1.0), dict(scale=NAN)):
        with pytest.raises(RuntimeError):
            sdpa_fwd_paged(**{**x, **bad})
    y = cuda(make(2, 4, 2, 1, [30, 600], 16, 64, 64, torch.bfloat16))
    with pytest.raises(RuntimeError):
        sdpa_fwd_paged(**y, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
