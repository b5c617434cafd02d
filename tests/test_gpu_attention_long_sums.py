"""Sums over very many keys with the same score, where every rounding has the same sign: lse and out against
the closed form.

The first key's score lies `gap` above the n - 1 others, which are equal, so lse = s0 + log(1 + (n - 1)
exp(-gap)), and with the same values at every key out is that value.  A row's sum may take 64 keys at a time,
32 terms a lane: 32 + n / 64 + 8 additions (the lanes and parts joined), each off by at most half a step, 2^-24
relative, and 10 more for the probabilities: the scores are exact (powers of two), their difference times
scale * log2(e) is rounded three times at most 4 in size, the exponential once.  lse takes 4 roundings of its own
size.  out: the same, a probability rounded to BF16, products added 16 keys at a time (steps of 2^-23, also where
they are cut off), and the result's rounding."""
import math

import pytest
import torch

import bit_microscaled_numerics_amd as nv
from parity import say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("gap", [0.75, 1.25, 1.625])
@pytest.mark.parametrize("rows,n", [(4, 65536), (66000, 65536), (66000, 262144)])
def test_equal_scores(rows, n, gap):
    """Few rows take their keys in parts, many rows one after the other."""
    say("attention equal scores", rows, n, gap)
    q, k = (torch.zeros(x, 1, 8, dtype=BF, device="cuda") for x in (rows, n))
    v = torch.full((n, 1, 8), 1.0, dtype=BF, device="cuda")
    q[..., 0] = 1.0
    k[0, 0, 0] = gap
    out, lse = nv.attention(q, k, v, scale=1.0)
    want = gap + math.log(1 + (n - 1) * math.exp(-gap))
    adds = 32 + n / 64 + 8 + 10
    tol = adds * 2.0 ** -24 + 4 * want * 2.0 ** -24
    assert float((lse.double() - want).abs().max()) <= tol
    tol = adds * 2.0 ** -24 + (n / 16 + 8) * 2.0 ** -23 + 2 * 2.0 ** -8
    assert float((out.double() - 1).abs().max()) <= tol
