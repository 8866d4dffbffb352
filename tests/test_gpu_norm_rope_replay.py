"""The norm and rotation captured into a graph and replayed on inputs that share
nothing with those of the capture: other rows, positions, weights, angles and cache
rows (the norm takes no notice of a row's scale, so scaled rows would show little).
"""
from __future__ import annotations

import pytest
import torch

from scaled_dot_product_06_gb300 import sdpa_qk_norm_rope, sdpa_qk_norm_rope_bwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,d_v,interleaved", [(64, 64, True), (128, 128, False), (192, 128, False)])
def test_other_inputs(d, d_v, interleaved):
    b, s, h, h_kv, rows, n_pos = 3, 40, 4, 2, 64, 500

    def make(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def r(*shape, dtype=torch.bfloat16):
            return torch.randn(*shape, generator=g, device="cuda").to(dtype)

        a = torch.rand(n_pos, d // 2, generator=g, device="cuda") * 6.28
        return {"q": r(b, s, h, d), "k": r(b, s, h_kv, d), "v": r(b, s, h_kv, d_v), "cos": a.cos(), "sin": a.sin(),
                "pos": torch.randint(0, n_pos, (b, s), generator=g, device="cuda").to(torch.int32),
                "wq": r(d, dtype=torch.float32), "wk": r(d, dtype=torch.float32),
                "at": torch.randint(0, rows - s + 1, (b,), generator=g, device="cuda").to(torch.int32),
                "dq": r(b, h, s, d), "dk": r(b, h_kv, s, d), "dv": r(b, h_kv, s, d_v),
                "kc": r(b, h_kv, rows, d), "vc": r(b, h_kv, rows, d_v)}

    def step(x):
        kw = dict(positions=x["pos"], q_weight=x["wq"], k_weight=x["wk"], interleaved=interleaved)
        f = sdpa_qk_norm_rope(x["q"], x["k"], x["cos"], x["sin"], v=x["v"], **kw)
        a = sdpa_qk_norm_rope(x["q"], x["k"], x["cos"], x["sin"], v=x["v"], kv_rows=x["at"], k_out=x["kc"],
                              v_out=x["vc"], **kw)
        g = sdpa_qk_norm_rope_bwd(x["dq"], x["dk"], x["q"], x["k"], x["cos"], x["sin"], dv_out=x["dv"], **kw)
        return (*f, *a, *g)

    x = make(1)
    first = [t.clone() for t in step(x)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x)
    for seed in (2, 3):
        y = make(seed)
        for n, t in x.items():
            t.copy_(y[n])
        graph.replay()
        torch.cuda.synchronize()
        want = step(y)
        assert all(torch.equal(p, w) for p, w in zip(out, want))
        assert not any(torch.equal(p, f) for p, f in zip(out, first))
