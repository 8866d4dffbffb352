"""Values that are infinite, not a number or very large in the attention over a paged
cache: they reach the elements of O that they are summed in, and nothing else."""
from __future__ import annotations

import pytest
import torch

from paged_exact import paged
from paged_ref import make
from scaled_dot_product_06_gb300 import sdpa_device_error, sdpa_fwd_paged
from scaled_dot_product_06_gb300.inputs import DTYPES

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
PAGE = 16

# (h, h_kv, lengths, d, d_v, dtype)
CASES = [
    (8, 2, [300, 77], 64, 64, "bf16"),                 # whole units, a tile or more
    (8, 2, [300, 77], 128, 128, "fp16"),
    (40, 1, [130, 400], 64, 64, "fp16"),               # halves of the rows
    (16, 1, [20000], 192, 128, "bf16"),                # joined by a kernel of its own
    (8, 1, [900] * 76 + [9000] * 4, 64, 64, "fp16"),   # joined by who leaves the last part
]


def call(x, **kw):
    got = sdpa_fwd_paged(**{n: t.cuda() for n, t in x.items()}, **kw)
    torch.cuda.synchronize()
    assert sdpa_device_error() == 0
    return got


def at(x, i, j):
    """Page and row of key j of sequence i."""
    return int(x["block_table"][i, j // PAGE]), j % PAGE


@pytest.mark.parametrize("c", CASES, ids=lambda c: f"h{c[0]}kv{c[1]}n{c[2][0]}d{c[3]}-{c[5]}")
def test_infinite_values(c):
    h, h_kv, lens, d, d_v, t = c
    x = make(len(lens), h, h_kv, 1, lens, PAGE, d, d_v, DTYPES[t], q_mul=1.0)
    clean = call(x)
    i, group = len(lens) - 1, h // h_kv
    n = lens[i]
    y = dict(x, v_pages=x["v_pages"].clone())
    last = n - 1
    # column: its keys with their values, and what O is then
    for col, keys, want in ((0, {0: INF}, INF), (1, {last: -INF}, -INF), (5, {n // 2: INF}, INF),
                            (6, {j: INF for j in range(0, n, 3)}, INF), (9, {0: INF, last: -INF}, NAN),
                            (11, {n // 3: NAN}, NAN), (13, {last: NAN, 0: INF}, NAN)):
        for j, f in keys.items():
            y["v_pages"][at(y, i, j)[0], 0, at(y, i, j)[1], col] = f
        clean[0][i, :group, 0, col] = want
    got = call(y)
    assert torch.equal(got[1], clean[1])
    assert torch.equal(torch.isnan(got[0]), torch.isnan(clean[0]))
    assert torch.equal(got[0].nan_to_num(7.0, INF, -INF), clean[0].nan_to_num(7.0, INF, -INF))


@pytest.mark.parametrize("score", [41.0, -41.0, 0.0])
def test_the_largest_finite_values(score):
    """bf16 values of v with keys * |v| < 2^67, where all scores are as far from 0 as leaves
    the first maximum at 0: 2^59 in the exponentials."""
    n, d = 500, 64
    q, k = torch.zeros(1, 2, 1, d).bfloat16(), torch.zeros(1, n, d).bfloat16()
    q[..., 0], k[..., 0] = 8.0, score  # q k / 8
    v = torch.full((1, n, d), 2.0 ** 58).bfloat16()
    v[:, :, 1::2] *= -1
    o, lse = call(paged(q, [k], [v], PAGE))
    assert torch.equal(o.cpu(), v[:, :1].expand(1, 2, d).reshape(1, 2, 1, d))
    assert (lse.cpu() - (float(k[0, 0, 0]) + torch.tensor(float(n)).log())).abs().max() < 2.0 ** -15
