"""GPU: rotations of more tokens than most calls hold."""
import math

import pytest
import torch

import speculative_decoding_medusa_b200 as M

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_token_counts_up_to_the_limit_of_an_int():
    """T = 2^31 - 1 tokens of one head of two elements, in place, on an odd
    element (nothing wider than an element fits): 8.6 GB of q, 8.6 of positions."""
    T = 2 ** 31 - 1
    flat = torch.empty(2 * T + 1, dtype=torch.bfloat16, device=DEV)
    flat.fill_(0.75)
    flat[1::2] = 0.5
    q = flat[1:].view(T, 1, 2)  # pairs (0.5, 0.75)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    M.medusa_rope(M.Rope(2, theta=10.0), q, None, pos, q, None)
    torch.cuda.synchronize()
    assert float(flat[0]) == 0.75
    # frequency 1: the angle is the position
    for lo in (0, 1 << 20, (1 << 30) + 77, T - 600000, T - 3000):
        hi = min(lo + 3000, T)
        a = torch.arange(lo, hi, dtype=torch.float64, device=DEV)
        c, s = a.cos(), a.sin()
        ref = torch.stack([0.5 * c - 0.75 * s, 0.5 * s + 0.75 * c], dim=-1)
        # angles to 2^-28 turns, cos, sin and products in fp32 (below 2^-20 of the
        # pair's 0.91), then half a step of bf16, 2^-8 of the result; the fp64
        # angle above is exact
        err = (q[lo:hi, 0].double() - ref).abs()
        assert bool((err <= 2.0 ** -8 * ref.abs() + 2.0 ** -19).all()), (lo, float(err.max()))
    # every token was turned, once: the pairs keep their length
    n, worst = 0, 0.0
    for lo in range(0, T, 1 << 28):
        x = q[lo:lo + (1 << 28), 0].float()
        length = (x * x).sum(-1)
        worst = max(worst, float((length - 0.8125).abs().max()))
        n += x.shape[0]
    # each element off by 2^-8 relative and 2^-19: the sum of squares by less
    # than 2 * 2^-8 * 0.8125 + 2^-16
    assert n == T and worst <= 2 * 2.0 ** -8 * 0.8125 + 2.0 ** -15, worst
    one = math.sqrt(0.8125)
    assert bool((q[-5000:, 0].float().norm(dim=-1) - one).abs().max() < 2.0 ** -7)
