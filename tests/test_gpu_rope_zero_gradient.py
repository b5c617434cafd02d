"""Rows of queries and keys whose incoming gradient is all zero (tokens that belong to no sequence)
take no part in the gradient of the norm and rotation, whatever they hold."""
import pytest
import torch

import bit_microscaled_numerics_amd as nv
from parity import say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

CASES = [  # T, Hq, Hkv, D, rot: whole pieces and single values, 1 to 64 lanes a row
    (40, 4, 2, 64, 64), (33, 3, 1, 22, 10), (9, 5, 5, 512, 512), (130, 2, 1, 8, 8), (70, 6, 2, 80, 36),
    (5, 2, 2, 250, 0), (300, 1, 3, 128, 128)]


def _call(T, Hq, Hkv, D, rot, dt, il, g):
    q, k, dq, dk = (torch.randn(T, H, D, generator=g).to(dt).cuda() for H in (Hq, Hkv, Hq, Hkv))
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=g)).cuda() for _ in range(2))
    at = (torch.arange(T, device="cuda"), (1e4 ** (-torch.arange(0, rot, 2) / max(rot, 1))).float().cuda())
    return q, k, dq, dk, wq, wk, *(at if rot else (None, None))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", CASES)
def test_rows_without_a_gradient(T, Hq, Hkv, D, rot, dt, il, value):
    """The same bits as with finite values in their place: such a row adds zeros to the sums."""
    say("rope zero gradient", T, Hq, Hkv, D, rot, dt, il, value)
    g = torch.Generator().manual_seed(T + D)
    q, k, dq, dk, wq, wk, pos, inv = _call(T, Hq, Hkv, D, rot, dt, il, g)
    hide_q, hide_k = torch.rand(T, Hq, generator=g).cuda() < 0.3, torch.rand(T, Hkv, generator=g).cuda() < 0.3
    hide_q[T - 1], hide_k[T - 1], hide_q[0, 0], hide_k[0, 0] = True, True, False, False
    dq[hide_q], dk[hide_k] = 0.0, 0.0
    want = nv.qk_norm_rope_grad(dq, dk, q, k, wq, wk, pos, inv, interleaved=il)
    assert all(torch.isfinite(x).all() for x in want)
    q[hide_q], k[hide_k] = value, value
    q[T - 1], k[T - 1] = 1.0, -1.0   # and one value of a row alone
    q[T - 1, :, D - 1], k[T - 1, :, 0] = value, value
    got = nv.qk_norm_rope_grad(dq, dk, q, k, wq, wk, pos, inv, interleaved=il)
    assert not got[0][hide_q].any() and not got[1][hide_k].any()
    for name, a, b in zip(("dq", "dk", "dq_weight", "dk_weight"), got, want):
        assert torch.equal(a, b), name


def test_rows_with_a_gradient_are_not_left_out():
    """One value of a row's gradient that is not zero, or is NaN, and the row counts."""
    say("rope one gradient")
    g = torch.Generator().manual_seed(1)
    q, k, dq, dk, wq, wk, pos, inv = _call(20, 2, 1, 64, 64, BF, False, g)
    dq.zero_()
    dq[3, 1, 63] = 2.0 ** -100
    q[3, 1, 5] = float("nan")
    got = nv.qk_norm_rope_grad(dq, dk, q, k, wq, wk, pos, inv)
    assert torch.isnan(got[0][3, 1]).all() and torch.isnan(got[2]).any()
    assert not got[0][3, 0].any() and not got[0][4].any()
    q[3, 1, 5] = 1.0
    dq[3, 1, 63] = float("nan")
    got = nv.qk_norm_rope_grad(dq, dk, q, k, wq, wk, pos, inv)
    assert torch.isnan(got[0][3, 1]).all() and torch.isnan(got[2]).any()


def test_no_row_with_a_gradient():
    say("rope no gradient")
    g = torch.Generator().manual_seed(2)
    q, k, dq, dk, wq, wk, pos, inv = _call(50, 3, 1, 48, 32, BF, True, g)
    nan = torch.full_like
    got = nv.qk_norm_rope_grad(dq.zero_(), dk.zero_(), nan(q, float("nan")), nan(k, float("nan")), wq, wk, pos, inv)
    assert not any(x.any() for x in got)
