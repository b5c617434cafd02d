"""Queries that see one key: their probability is 1 whatever their score, so ds, dq and what they add to dk are
exactly 0, and out and dv's part are the value and the gradient themselves."""
import pytest
import torch

import attn_reference as ref
import bit_microscaled_numerics_amd as nv
from parity import say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _rand(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(BF).cuda()


def _close(got, want, tol, name):
    bad = (got.double() - want).abs() > tol
    assert not (bad & (got.double() != want)).any(), (name, int(bad.sum()))


def _check(g, Tq, Tk, Hq, Hkv, D, causal, window, cu=None):
    q, k, v, dout = (_rand(g, T, H, D) for T, H in ((Tq, Hq), (Tk, Hkv), (Tk, Hkv), (Tq, Hq)))
    kw = dict(causal=causal, window=window)
    bounds = [(0, Tq, 0, Tk)]
    if cu is not None:
        kw.update(cu_q=torch.tensor(cu[0], device="cuda"), cu_k=torch.tensor(cu[1], device="cuda"))
        bounds = list(zip(cu[0], cu[0][1:], cu[1], cu[1][1:]))
    out, lse = nv.attention(q, k, v, **kw)
    dq, dk, dv = nv.attention_grad(dout, q, k, v, out, lse, **kw)
    seen = torch.zeros(Tq, Tk, dtype=torch.bool)
    for a, b, c, d in bounds:
        seen[a:b, c:d] = ref.seen_mask(b - a, d - c, causal, window)
    alone = (seen.sum(1) == 1).cuda()
    assert alone.any()
    at = seen.int().argmax(1).cuda()[alone]
    assert torch.equal(out[alone], v[at].repeat_interleave(Hq // Hkv, 1))
    assert not dq[alone].any()
    only = ~seen[~alone.cpu()].any(0).cuda()   # keys that no other query sees
    assert not dk[only].any()
    r, t = ref.attention(q, k, v, D ** -0.5, causal, window, bounds, dout)
    for name, x in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, dq, dk, dv)):
        _close(x, r[name], t[name], name)


@pytest.mark.parametrize("Tq,Tk,Hq,Hkv,causal,window", [
    (1, 1, 1, 1, False, 0), (1, 1, 8, 2, True, 0), (5000, 1, 2, 1, False, 0), (70, 1, 3, 3, False, 0),
    (40, 1, 4, 1, True, 0), (300, 300, 4, 2, True, 1), (33, 700, 2, 1, True, 1), (400, 300, 2, 2, True, 1),
    (130, 130, 6, 1, True, 0), (257, 200, 5, 1, True, 0), (100, 64, 2, 1, True, 7)])
@pytest.mark.parametrize("D", [64, 80, 128])
def test_one_key(Tq, Tk, Hq, Hkv, D, causal, window):
    say("attention one key", Tq, Tk, Hq, Hkv, D, causal, window)
    _check(torch.Generator().manual_seed(Tq + Tk), Tq, Tk, Hq, Hkv, D, causal, window)


@pytest.mark.parametrize("nq,nk", [
    ([1] * 200, [1] * 200), ([3, 1, 50, 1, 90], [1, 1, 50, 30, 1]), ([0, 5, 64, 7], [1, 1, 0, 1]),
    ([40, 2, 200], [1, 90, 130])])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 1), (True, 5)])
def test_one_key_packed(nq, nk, causal, window):
    say("attention one key packed", nq[:5], nk[:5], causal, window)
    cu = [[sum(n[:i]) for i in range(len(n) + 1)] for n in (nq, nk)]
    _check(torch.Generator().manual_seed(len(nq)), sum(nq), sum(nk), 4, 2, 64, causal, window, cu)


def test_not_finite_stays():
    """p (dp - delta) is NaN where the one value or its gradient is not finite."""
    say("attention one key not finite")
    g = torch.Generator().manual_seed(3)
    for which in range(4):
        q, k, v, dout = (_rand(g, 9, H, 64) for H in (2, 1, 1, 2))
        (q, k, v, dout)[which][4, 0, 7] = float("nan")
        out, lse = nv.attention(q, k, v, causal=True, window=1)
        dq, dk, _ = nv.attention_grad(dout, q, k, v, out, lse, causal=True, window=1)
        assert torch.isnan(dq[4, 0]).all() and torch.isnan(dk[4]).all()
        assert not dq[torch.arange(9) != 4].any() and not dk[torch.arange(9) != 4].any()
