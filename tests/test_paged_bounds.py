"""That the bounds of paged_exact tell the attention's arithmetic from coarser ones:
the kernel's roundings, repeated in plain operations on the CPU, stay inside; with P
rounded once to 16 bits, or with the coarser tanh, they do not."""
import numpy as np
import pytest
import torch

from paged_exact import bounds, cancelling, weights

SIZES = [(2, 8, 64, 64, 64), (1, 16, 100, 128, 128), (1, 32, 64, 192, 128), (1, 64, 96, 64, 64)]


def rounded(s, v, t, parts):
    """O in the kernel's roundings: P of the largest score (fp16) or of 0 (bf16) in one
    16-bit part or two, fp32 sums."""
    y = torch.from_numpy(s * np.log2(np.e)).float()
    m = y.max(-1, keepdim=True).values if t == torch.float16 else torch.zeros(1)
    p = torch.exp2(y - m)
    high = p.to(t).float()
    used = high if parts == 1 else high + ((p - high) * 2.0 ** 18).to(t).float() * 2.0 ** -18 \
        if t == torch.float16 else high + (p - high).to(t).float()
    o = used.double().numpy() @ v / p.sum(-1, keepdim=True).double().numpy()
    return torch.from_numpy(o).to(t).double().numpy()


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_one_part_of_p_is_seen(size, t):
    q, k, v = cancelling(*size, t, seed=1)
    s, w = weights(q, k, size[3] ** -0.5)
    assert np.abs(s).max() * np.log2(np.e) < 32
    o, _, oe, _ = bounds(s, w, v.double().numpy(), t)
    assert (np.abs(rounded(s, v.double().numpy(), t, 2) - o) <= oe).all()
    over = np.abs(rounded(s, v.double().numpy(), t, 1) - o) > oe
    # most of the values that nearly cancel, and so in any test of some dozens of them
    r = size[1]
    assert np.mean([over[:, e, e::r].mean() for e in range(r)]) > 0.6


def capped_bound(s, cap):
    """LSE of one key: the capped score itself. Its argument is rounded three times (2^-24
    each), the tanh is good to 2^-22 of itself, the factor rounded twice; then the
    exponential and the logarithm: 2^-22 and, of a number of its size, 2^-21."""
    y = np.abs(cap * np.tanh(s / cap))
    return y * (5 * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -21) + 2.0 ** -21


@pytest.mark.parametrize("cap", [50.0, 1000.0])
def test_the_coarser_tanh_is_seen(cap):
    s = np.linspace(-2, 2, 1999)
    z = torch.from_numpy(s / cap).float()
    want = cap * np.tanh(s / cap)
    fine = (torch.tanh(z) * cap).double().numpy()
    assert (np.abs(fine - want) <= capped_bound(s, cap)).all()
    coarse = (cap - 2 * cap / (1 + torch.exp(2 * z))).double().numpy()
    assert (np.abs(coarse - want) > capped_bound(s, cap)).mean() > 0.1
