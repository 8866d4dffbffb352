"""Calls on streams that are not the current one: what a call allocates is neither in
use elsewhere when it runs nor given away before it has run. Streams are kept
busy by ordinary products, so that host and device are apart when it matters.
"""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

from scaled_dot_product_06_gb300 import (sdpa_bwd, sdpa_bwd_varlen, sdpa_device_error, sdpa_dropout_mask, sdpa_fwd,
                                         sdpa_fwd_prefix, sdpa_fwd_prefix_workspace_size,
                                         sdpa_qk_norm_rope, sdpa_qk_norm_rope_bwd)

pytestmark = pytest.mark.gpu


def rand(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


# b180: more work items than CTAs, which are then handed out by a counter in the workspace
B, H, D, S_P, S_MAX = 180, 4, 64, 300, 500


def prefix_call(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = torch.randint(1, S_MAX + 1, (B,), generator=g, device="cuda").to(torch.int32)
    args = (rand(g, B, H, 1, D), rand(g, 1, S_P, D), rand(g, 1, S_P, D), rand(g, B, 1, S_MAX, D),
            rand(g, B, 1, S_MAX, D), n)
    return lambda **kw: sdpa_fwd_prefix(*args, softcap=30.0, **kw)


def norm_call(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k = rand(g, 2, 700, 8, 128), rand(g, 2, 700, 2, 128)
    dy, dk, w = rand(g, 2, 8, 700, 128), rand(g, 2, 2, 700, 128), rand(g, 128, dtype=torch.float32)

    def run(**kw):
        a = sdpa_qk_norm_rope(q, k, None, None, v=k, q_weight=w, k_weight=w, **kw)
        r = sdpa_qk_norm_rope_bwd(dy, dk, q, k, None, None, q_weight=w, k_weight=w, **kw)
        return (*a, *(x for x in r if x is not None))
    return run


def attention_call(softcap):
    def make(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        q, k, v, do = (rand(g, 2, h, 384, 128) for h in (4, 2, 2, 4))

        def run(**kw):
            c = dict(is_causal=True, softcap=softcap, **kw)
            o, lse = sdpa_fwd(q, k, v, **c)
            return (o, lse, *sdpa_bwd(q, k, v, o, do, lse, deterministic=True, **c)[:3])
        return run
    return make


def packed_call(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, do = (rand(g, h, 500, 64) for h in (4, 2, 2, 4))
    o, lse = rand(g, 4, 500, 64), rand(g, 4, 500, dtype=torch.float32) + 6
    st = torch.tensor([0, 100, 333, 500], dtype=torch.int32, device="cuda")
    return lambda **kw: sdpa_bwd_varlen(q, k, v, o, do, lse, st, st, 233, 233, is_causal=True, softcap=20.0,
                                        deterministic=True, **kw)


CALLS = {"prefix": prefix_call, "norm": norm_call, "capped": attention_call(20.0), "plain": attention_call(None),
         "packed": packed_call}


@pytest.fixture(scope="module")
def busy():
    a = torch.randn(4096, 4096, device="cuda").bfloat16()

    def occupy(stream, n=60):  # some milliseconds
        with torch.cuda.stream(stream):
            c = torch.empty_like(a)
            for _ in range(n):
                torch.mm(a, a, out=c)
            return c
    return occupy


def overwrite():
    """Every kind of block that the current stream's allocator has free, filled."""
    held = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x7F)
            for k in range(9, 25) for n in (1 << k, 3 << (k - 1))]
    return held


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want)) and len(got) == len(want)


@pytest.mark.parametrize("name", CALLS)
def test_two_streams_at_once(name, busy):
    one, two = CALLS[name](1), CALLS[name](2)
    want = [[t.clone() for t in f()] for f in (one, two)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        kept = [busy(s1), busy(s2)]
        got = [one(stream=s1)]
        kept.append(overwrite())
        got += [two(stream=s2), one(stream=s1)]
        kept.append(overwrite())
        got += [two(stream=s2)]
        torch.cuda.synchronize()
        for i, r in enumerate(got):
            assert same(r, want[i % 2]), i
        del kept, got
    assert sdpa_device_error() == 0


def test_two_streams_with_a_workspace_each(busy):
    one, two = prefix_call(1), prefix_call(2)
    want = [[t.clone() for t in f()] for f in (one, two)]
    size = sdpa_fwd_prefix_workspace_size(B, H, 1, 1, S_P, S_MAX, D, D)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = [busy(s1), busy(s2)]  # both queues fill before either begins
    got = [(one(stream=s1, workspace=ws[0]), two(stream=s2, workspace=ws[1])) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(same(a, want[0]) and same(b, want[1]) for a, b in got)
    assert sdpa_device_error() == 0
    del kept


@pytest.mark.parametrize("name", CALLS)
def test_outputs_are_not_memory_in_use(name, busy):
    """Tensors dropped while the current stream still reads them are not the outputs
    of a call on an idle stream, nor are its outputs, dropped likewise, the next's."""
    run, other = CALLS[name](3), CALLS[name](4)
    want = [t.clone() for t in run()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    main = torch.cuda.current_stream()
    for _ in range(3):
        old = [torch.full_like(t, 3.0) for t in want]
        kept = busy(main)
        read = [t + 1 for t in old]
        del old
        got = run(stream=s)
        s.synchronize()
        copies = [t.clone() for t in got]  # behind the busy work, on the current stream
        del got
        again = other(stream=s)
        torch.cuda.synchronize()
        assert all((t == 4).all() for t in read)
        assert same(copies, want)
        del kept, again
    assert sdpa_device_error() == 0


def test_captured_on_a_side_stream():
    """A call on a stream that has joined a capture: its memory is the graph's."""
    run = prefix_call(5)
    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    run(stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = run(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        held = overwrite()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want)
        del held
    assert sdpa_device_error() == 0


def test_keep_bits_on_another_stream(busy):
    want = sdpa_dropout_mask(2, 4, 96, 128, 0.3, 5, 6)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = busy(s)
    got = sdpa_dropout_mask(2, 4, 96, 128, 0.3, 5, 6, stream=s)
    held = overwrite()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del kept, held


def test_foreign_stream_object():
    """A stream of another library: an object with a handle."""
    s = torch.cuda.Stream()
    run = attention_call(20.0)(6)
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    got = run(stream=SimpleNamespace(cuda_stream=s.cuda_stream))
    torch.cuda.synchronize()
    assert same(got, want)
