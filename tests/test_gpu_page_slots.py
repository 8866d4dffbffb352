"""Block tables and slot maps (sdpa_page_slots) against the plain form, whole
numbers equal; in place, captured and replayed, on another stream."""
from __future__ import annotations

import random

import pytest
import torch

from paged_ref import ceil, page_slots
from scaled_dot_product_06_gb300 import sdpa_page_slots

pytestmark = pytest.mark.gpu


def case(rng, b, page, longest, wide, free, ended=0.2, fresh=False, most=5, bad=False):
    """(lens, new, table, ring, span): a consistent pool, or numbers of any kind."""
    n = [0 if fresh else rng.randrange(0, longest + 1) for _ in range(b)]
    x = [-1 if rng.random() < ended else rng.randrange(0, most + 1) for _ in range(b)]
    have = [min(ceil(v, page), wide) for v in n]
    pool = sum(have) + free + 1
    order = list(range(pool))
    rng.shuffle(order)
    table, at = [], 0
    for k in have:
        table.append(order[at:at + k] + [-1] * (wide - k))
        at += k
    ring = list(order)
    head = rng.randrange(0, 5 * pool)
    for i in range(free):
        ring[(head + i) % pool] = order[at + i]
    if bad:
        for r in table:
            for c in range(wide):
                if rng.random() < 0.2:
                    r[c] = rng.choice((-5, pool, 1 << 30, -(1 << 31)))
        n[rng.randrange(b)] = -7
    return n, x, table, ring, [head, head + free]


def cuda(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def call(n, x, table, ring, span, page, **kw):
    wide = len(table[0]) if table else 0
    t = cuda(table).view(len(table), wide)
    r = cuda(ring)
    got = sdpa_page_slots(cuda(n), cuda(x), t, r, cuda(span, torch.int64), page, **kw)
    return (*got, t, r)


def check(got, want):
    for name, a, b in zip(("slots", "positions", "starts", "seqlens", "range", "table", "ring"), got, want):
        if b is None:
            assert a is None, name
            continue
        b = torch.tensor(b, dtype=a.dtype).view(a.shape) if a.numel() else torch.empty(a.shape, dtype=a.dtype)
        assert torch.equal(a.cpu(), b), (name, (a.cpu() != b).nonzero()[:4].tolist())


# b, page, longest, free pages, most new tokens a request, packed rows (None: padded), padded width
CASES = [
    (1, 16, 0, 1, 1, None, 1),
    (1, 1, 9, 20, 5, 5, None),
    (7, 16, 100, 40, 5, None, 5),
    (7, 16, 100, 2, 50, None, 50),          # too few pages
    (33, 8, 300, 100, 1, 40, None),
    (33, 8, 300, 100, 60, 700, None),       # too few entries
    (256, 16, 4096, 256, 1, None, 1),
    (300, 24, 50, 900, 70, 9001, None),     # pages of no power of two, a cluster of CTAs
    (1000, 32, 200, 500, 20, 20000, None),
    (1024, 16, 64, 0, 3, None, 3),          # no free page
    (1025, 16, 64, 60, 3, 2000, None),      # two chunks of requests
    (3000, 16, 64, 400, 9, None, 9),
    (2500, 4, 30, 3000, 9, 30000, None),
    (5, 64, 10000, 2000, 40000, 131072, None),
]


@pytest.mark.parametrize("bad", [False, True])
@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_matches_plain_form(c, bad):
    b, page, longest, free, most, rows, width = c
    rng = random.Random(b * 31 + page)
    for fresh in (False, True):
        wide = ceil(longest + most, page) + rng.randrange(0, 2) - (1 if b > 5 and longest > page else 0)
        x = case(rng, b, page, longest, max(wide, 1), free, fresh=fresh, most=most, bad=bad)
        check(call(*x, page, rows=rows, width=width), page_slots(*x, page, rows=rows, width=width))


def test_no_requests_and_no_pages():
    check(call([], [], [], [3, 1], [5, 6], 16, rows=6), ([-1] * 6, [0] * 6, [0], [], [5, 6], [], [3, 1]))
    check(call([], [], [], [3, 1], [5, 6], 16, width=2), ([], [], None, [], [5, 6], [], [3, 1]))
    got = call([0, 3], [2, 0], [[-1], [-1]], [], [0, 0], 16, rows=3)
    check(got, ([-1] * 3, [0, 1, 0], [0, 2, 2], [0, 3], [0, 0], [[-1], [-1]], []))
    # an empty tensor of entries, lengths alone
    got = call([4, 5], [0, -1], [[1], [0]], [7, 7], [2, 2], 8, width=0)
    check(got, ([], [], None, [4, 0], [2, 3], [[1], [0]], [0, 7]))


def test_counters_of_any_kind_stay_inside():
    """Counters that no ring has: nothing outside the tensors is written."""
    big = torch.full((64,), 77, dtype=torch.int32, device="cuda")
    ring = big[16:24]
    for span in ([-5, 3], [1 << 62, (1 << 62) + 3], [9, 2], [-(1 << 63), (1 << 63) - 1], [0, 1 << 40]):
        t = cuda([[0, 1, 2, 3], [4, 5, 6, 7], [1, 1, 1, 1]])
        got = sdpa_page_slots(cuda([100, 60, 3]), cuda([5, -1, 60]), t, ring, cuda(span, torch.int64), 16, width=70)
        torch.cuda.synchronize()
        assert (big[:16] == 77).all() and (big[24:] == 77).all()
        assert got[3].tolist()[:2] == [100, 0]
        s = got[0]
        assert ((s >= -1) & (s < 128)).all()


def test_given_outputs_and_their_neighbours():
    """Outputs in the middle of larger buffers; a table that is part of a wider one."""
    rng = random.Random(5)
    x = case(rng, 40, 16, 200, 14, 60, most=30)
    buf = {n: torch.full((k,), 99, dtype=torch.int32, device="cuda") for n, k in
           (("slots", 8 + 801), ("positions", 8 + 801), ("starts", 4 + 43), ("seqlens_out", 4 + 42))}
    tables = torch.full((40, 20), 55, dtype=torch.int32, device="cuda")
    tables[:, 3:17] = cuda(x[2])
    ring = cuda(x[3])
    out = {"slots": buf["slots"][4:805], "positions": buf["positions"][4:805], "starts": buf["starts"][4:45],
           "seqlens_out": buf["seqlens_out"][4:44]}
    got = sdpa_page_slots(cuda(x[0]), cuda(x[1]), tables[:, 3:17], ring, cuda(x[4], torch.int64), 16, rows=801, **out)
    assert got[0] is out["slots"] and got[2] is out["starts"]
    check((*got, tables[:, 3:17], ring), page_slots(*x, 16, rows=801))
    for n, t in buf.items():
        k = out[n].numel()
        assert (t[:4] == 99).all() and (t[4 + k:] == 99).all(), n
    assert (tables[:, :3] == 55).all() and (tables[:, 17:] == 55).all()


@pytest.mark.parametrize("b,rows", [(50, None), (50, 9000), (1500, None), (1500, 12000)])
def test_in_place_and_replayed(b, rows):
    """Lengths and counters advanced in place by a captured call, step after step,
    pages coming back and being given out again."""
    rng = random.Random(b)
    x = case(rng, b, 8, 40, 30, 6 * b, most=6)
    kw = {"rows": rows} if rows else {"width": 6}
    n, new, span = cuda(x[0]), cuda(x[1]), cuda(x[4], torch.int64)
    table, ring = cuda(x[2]), cuda(x[3])
    want = x
    g = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    kept = [t.clone() for t in (n, new, span, table, ring)]
    with torch.cuda.stream(stream):
        sdpa_page_slots(n, new, table, ring, span, 8, seqlens_out=n, free_range_out=span, **kw)
    torch.cuda.synchronize()
    for t, k in zip((n, new, span, table, ring), kept):
        t.copy_(k)
    with torch.cuda.graph(g):
        got = sdpa_page_slots(n, new, table, ring, span, 8, seqlens_out=n, free_range_out=span, **kw)
    assert got[3] is n and got[4] is span
    for step in range(12):
        step_new = [-1 if rng.random() < 0.15 else rng.randrange(0, 7) for _ in range(b)]
        new.copy_(cuda(step_new))
        g.replay()
        want = page_slots(want[0], step_new, want[2], want[3], want[4], 8, **kw)
        check((*got, table, ring), want)
        want = (want[3], None, want[5], want[6], want[4])


def test_another_stream():
    rng = random.Random(9)
    x = case(rng, 64, 16, 500, 40, 300, most=40)
    n, new, table, ring, span = cuda(x[0]), cuda(x[1]), cuda(x[2]), cuda(x[3]), cuda(x[4], torch.int64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sdpa_page_slots(n, new, table, ring, span, 16, rows=3001, stream=s)
    s.synchronize()
    check((*got, table, ring), page_slots(*x, 16, rows=3001))


def test_binding_refusals():
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    t, span = torch.zeros(4, 3, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    sdpa_page_slots(i, i, t, i, span, 16, width=1)
    for a, kw in (((i, i[:3], t, i, span, 16), dict(width=1)), ((i, i, t[:3], i, span, 16), dict(width=1)),
                  ((i, i, t.long(), i, span, 16), dict(width=1)), ((i, i, t, i, span.int(), 16), dict(width=1)),
                  ((i, i, t.t(), i, span, 16), dict(width=1)), ((i, i, t, i, span, 16), dict()),
                  ((i, i, t[:1].expand(4, 3), i, span, 16), dict(width=1)), ((i, i.cpu(), t, i, span, 16), dict(width=1)),
                  ((i, i, t, i, span, 16), dict(rows=4, width=1)), ((i, i, t, i, span, 16), dict(width=1, starts=i)),
                  ((i, i, t, i, span, 16), dict(width=1, slots=i)), ((i, i, t, i, span, 16), dict(rows=4, starts=i)),
                  ((i, i, t, i, span, 16), dict(rows=3, slots=torch.zeros(6, dtype=torch.int32, device="cuda")[::2]))):
        with pytest.raises(ValueError):
            sdpa_page_slots(*a, **kw)


def test_outputs_made_in_one_allocation_are_apart():
    """Each new output is contiguous, on its own bytes, and outlives the others."""
    lens = torch.tensor([5, 0, 40], dtype=torch.int32, device="cuda")
    new = torch.tensor([3, 2, 1], dtype=torch.int32, device="cuda")
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    ring = torch.arange(100, 150, dtype=torch.int32, device="cuda") % 50
    span = torch.tensor([0, 20], device="cuda")
    out = sdpa_page_slots(lens, new, table, ring, span, 16, rows=7)
    assert [tuple(t.shape) for t in out] == [(7,), (7,), (4,), (3,), (2,)]
    assert [t.dtype for t in out] == [torch.int32] * 4 + [torch.int64] and all(t.is_contiguous() for t in out)
    ends = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in out)
    assert all(a[1] <= b[0] for a, b in zip(ends, ends[1:]))
    want = [t.clone() for t in out]
    kept = out[2]
    for t in out[:2]:
        t.fill_(-7)
    assert all(torch.equal(t, w) for t, w in zip(out[2:], want[2:]))
    del out, t
    torch.empty(4096, device="cuda").fill_(3)
    assert torch.equal(kept, want[2])
    empty = sdpa_page_slots(lens, new, table, ring, span, 16, rows=0)
    assert empty[0].shape == (0,) and empty[3].tolist() == [5, 0, 40]
