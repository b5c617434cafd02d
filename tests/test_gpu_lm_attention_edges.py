"""SelfAttention against float64 autograd away from its defaults: without norms, adjacent pairs, both
directions, and calls at the edges of what it takes."""
import pytest
import torch

import attn_reference as ref
from bit_microscaled_numerics_amd import lm
from parity import say

pytestmark = pytest.mark.gpu
BF, HALF = torch.bfloat16, 2.0 ** -8


def _rand(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(BF).cuda()


def _near(got, want, rel):
    """Norm-wise: rounding errors of independent sign, each at most `rel` of its entry."""
    assert got.shape == want.shape
    assert (got.double() - want).norm() <= rel * want.norm()


def _reference(m, qkv, bounds, dout):
    """Float64 autograd of one row of tokens; (out, dqkv, and dq_weight, dk_weight if there are norms)."""
    heads, kv, D, eps, il, norm, scale, causal, window = m.how
    x = qkv.double().requires_grad_()
    w = [p.double().detach().requires_grad_() for p in (m.q_weight, m.k_weight)] if norm else []
    T, n = x.shape[0], m.inv_freq.numel()
    q, k, v = (y.view(T, -1, D) for y in x.split((heads * D, kv * D, kv * D), -1))
    pos = torch.cat([torch.arange(b - a) for a, b in bounds]).double().cuda()
    t = (pos.unsqueeze(1) * m.inv_freq.double()).unsqueeze(1)

    def turn(y, side):
        if norm:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w[side]
        pairs = y[..., :2 * n].unflatten(-1, (n, 2) if il else (2, n))
        a, b = pairs.unbind(-1 if il else -2)
        turned = torch.stack((a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()), -1 if il else -2)
        return torch.cat((turned.flatten(-2), y[..., 2 * n:]), -1)

    q, k = turn(q, 0), turn(k, 1)
    rows = []
    for a, b in bounds:
        seen = ref.seen_mask(b - a, b - a, causal, window, "cuda")
        for h in range(heads):
            z = (scale * q[a:b, h] @ k[a:b, h * kv // heads].T).masked_fill(~seen, -torch.inf)
            rows.append(torch.softmax(z, -1) @ v[a:b, h * kv // heads])
    out = torch.cat([torch.stack(rows[i * heads:(i + 1) * heads], 1) for i in range(len(bounds))])
    out = out.reshape(T, heads * D)
    return (out.detach(), *torch.autograd.grad((out * dout.double()).sum(), (x, *w)))


def _results(m, qkv, dout, **kw):
    x = qkv.detach().requires_grad_()
    out = m(x, **kw)
    params = list(m.parameters())
    return (out.detach(), *torch.autograd.grad(out, (x, *params), dout))


# Roundings to BF16 on the way: q and k after the norm and rotation (they move the scores by scale *
# sum |q||k| 2^-8 / sqrt(D), some 2^-8 of p), p, ds, the intermediate gradients and the results: six of
# independent sign, the most of each HALF of its entry.
REL = 6 ** 0.5 * HALF


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("il,rot", [(False, 32), (True, 32), (True, 20), (False, 0)])
@pytest.mark.parametrize("causal", [True, False])
def test_variants(norm, il, rot, causal):
    say("lm module variant", norm, il, rot, causal)
    g = torch.Generator().manual_seed(7)
    T, heads, kv, D = 130, 4, 2, 32
    m = lm.SelfAttention(heads, D, kv, rot=rot, norm=norm, interleaved=il, causal=causal, device="cuda")
    with torch.no_grad():
        for p in m.parameters():
            p.add_(_rand(g, D, std=0.2))
    qkv, dout = _rand(g, T, (heads + 2 * kv) * D), _rand(g, T, heads * D)
    cu = torch.tensor([0, 50, T], dtype=torch.int32, device="cuda")
    got = _results(m, qkv, dout, cu=cu)
    want = _reference(m, qkv, [(0, 50), (50, T)], dout)
    assert len(got) == len(want)
    for a, b in zip(got, want):
        _near(a, b, REL)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("before", [0, 5])
def test_tokens_of_no_sequence_reach_nothing(before, value):
    """Rows before the first and behind the last sequence hold what was there: neither the other rows'
    results nor the gradients of the norms' weights take it over; their own are zeros."""
    say("lm module padding", before, value)
    g = torch.Generator().manual_seed(8)
    T, extra, heads, kv, D = 150, 11, 4, 2, 32
    m = lm.SelfAttention(heads, D, kv, device="cuda")
    qkv, dout = _rand(g, before + T + extra, (heads + 2 * kv) * D), _rand(g, before + T + extra, heads * D)
    real = slice(before, before + T)
    none = torch.ones(before + T + extra, dtype=torch.bool, device="cuda")
    none[real] = False
    qkv[none] = value
    cu = torch.tensor([before, before + 60, before + T], dtype=torch.int32, device="cuda")
    out, dqkv, dwq, dwk = _results(m, qkv, dout, cu=cu)
    assert not out[none].any() and not dqkv[none].any()
    want = _reference(m, qkv[real], [(0, 60), (60, T)], dout[real])
    for a, b in zip((out[real], dqkv[real], dwq, dwk), want):
        _near(a, b, REL)


@pytest.mark.parametrize("cast", [lambda m: m.to(BF), lambda m: m.bfloat16().float(), lambda m: m.cpu().half().float().cuda()])
def test_module_that_was_cast(cast):
    """Positions in the tens of thousands: frequencies with fewer bits would turn rows elsewhere."""
    say("lm module cast")
    g = torch.Generator().manual_seed(9)
    qkv, pos = _rand(g, 90, 6 * 32), 50000 + torch.arange(90, device="cuda")
    want = lm.SelfAttention(2, 32, device="cuda")(qkv, positions=pos)
    assert torch.equal(cast(lm.SelfAttention(2, 32, device="cuda"))(qkv, positions=pos), want)


@pytest.mark.parametrize("shape", [(0,), (2, 0), (0, 3)])
@pytest.mark.parametrize("norm,rot", [(True, 32), (False, 0)])
def test_no_tokens(shape, norm, rot):
    """As the functions below: results without rows, gradients of the weights that are zero."""
    say("lm module no tokens", shape, norm, rot)
    m = lm.SelfAttention(4, 32, 2, norm=norm, rot=rot, device="cuda")
    calls = [dict()] + [dict(cu=torch.zeros(n, dtype=torch.int32, device="cuda")) for n in (1, 3) if len(shape) == 1]
    for kw in calls:
        out, dqkv, *dw = _results(m, torch.zeros(*shape, 256, dtype=BF, device="cuda"),
                                  torch.zeros(*shape, 128, dtype=BF, device="cuda"), **kw)
        assert out.shape == (*shape, 128) and dqkv.shape == (*shape, 256)
        assert len(dw) == (2 if norm else 0) and not any(x.any() for x in dw)


def test_windows_over_one_row_of_tokens():
    say("lm module windows")
    g = torch.Generator().manual_seed(10)
    m = lm.SelfAttention(4, 32, 2, device="cuda")
    tokens, dout = _rand(g, 50, 256), _rand(g, 7, 20, 128)
    windows = tokens.unfold(0, 20, 5).transpose(1, 2)
    for a, b in zip(_results(m, windows, dout), _results(m, windows.contiguous(), dout)):
        assert torch.equal(a, b)
