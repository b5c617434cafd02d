"""The torch layer of attention and of the norm and rotation: autograd against the functional
forms and against float64 autograd of the definitions, layouts, packed sequences, graphs, and the
example that trains with them."""
import importlib.util
import math
import os

import pytest
import torch

import attn_reference as ref
import bit_microscaled_numerics_amd as nv
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


@pytest.mark.parametrize("kind", ["plain", "expanded", "odd_start", "heads_first"])
def test_attention_gradients_are_the_functional_ones(kind):
    say("lm attention", kind)
    g = torch.Generator().manual_seed(1)
    B, T, Hq, Hkv, D = 2, 75, 4, 2, 40
    q, k, v = (_rand(g, B, T, H, D) for H in (Hq, Hkv, Hkv))
    out, lse = nv.attention(q, k, v, causal=True)
    dout = _rand(g, B, T, Hq, D)
    if kind == "expanded":
        dout = dout[..., :1].expand(B, T, Hq, D)
    want = nv.attention_grad(dout.contiguous(), q, k, v, out, lse, causal=True)
    args = []
    for x in (q, k, v):
        if kind == "odd_start":
            flat = torch.zeros(x.numel() + 3, dtype=BF, device="cuda")
            flat[3:].copy_(x.reshape(-1))
            x = flat[3:].view_as(x)
        elif kind == "heads_first":
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        args.append(x.detach().requires_grad_())
    got = lm.attention(*args, causal=True)
    assert torch.equal(got, out)
    got.backward(dout)
    for x, w in zip(args, want):
        assert torch.equal(x.grad, w)
    with torch.no_grad():
        assert torch.equal(lm.attention(*args, causal=True), out)


def test_one_side_frozen():
    g = torch.Generator().manual_seed(2)
    q, k, v = (_rand(g, 30, H, 16) for H in (2, 1, 1))
    v.requires_grad_()
    out = lm.attention(q, k, v)
    out.backward(torch.ones_like(out))
    assert q.grad is None and k.grad is None and v.grad is not None


@pytest.mark.parametrize("shape", [(50,), (2, 25), ()])
@pytest.mark.parametrize("il", [False, True])
def test_norm_and_rotation(shape, il):
    say("lm rope", shape, il)
    g = torch.Generator().manual_seed(3)
    q, k = _rand(g, *shape, 3, 24).requires_grad_(), _rand(g, *shape, 1, 24).requires_grad_()
    wq, wk = (torch.nn.Parameter(1 + 0.1 * torch.randn(24, generator=g).cuda()) for _ in range(2))
    inv = (1e4 ** (-torch.arange(0, 16, 2) / 16)).float().cuda()
    pos = torch.arange(shape[-1], device="cuda") if shape else torch.tensor(7, device="cuda")
    a, b = lm.qk_norm_rope(q, k, wq, wk, pos, inv, interleaved=il)
    n = math.prod(shape)
    flat = [x.detach().reshape(n, *x.shape[-2:]) for x in (q, k)]
    at = pos.expand(shape).reshape(-1).contiguous()
    fa, fb = nv.qk_norm_rope(*flat, wq.detach(), wk.detach(), at, inv, interleaved=il)
    assert torch.equal(a.reshape(fa.shape), fa) and torch.equal(b.reshape(fb.shape), fb)
    da, db = _rand(g, *a.shape), _rand(g, *b.shape)
    torch.autograd.backward((a, b), (da, db))
    want = nv.qk_norm_rope_grad(da.reshape(fa.shape), db.reshape(fb.shape), *flat, wq.detach(), wk.detach(), at,
                                inv, interleaved=il)
    for x, w in zip((q, k, wq, wk), want):
        assert torch.equal(x.grad.reshape(w.shape), w)


def _module_reference(m, qkv, bounds, dout):
    """Float64 autograd of SelfAttention on one row of tokens."""
    heads, kv, D, eps, il, norm, scale, causal, window = m.how
    x = qkv.double().requires_grad_()
    w = [p.double().detach().requires_grad_() for p in (m.q_weight, m.k_weight)]
    T = x.shape[0]
    q, k, v = (y.view(T, -1, D) for y in x.split((heads * D, kv * D, kv * D), -1))
    pos = torch.cat([torch.arange(b - a) for a, b in bounds]).double().cuda()
    inv = m.inv_freq.double()
    t = (pos.unsqueeze(1) * inv).unsqueeze(1)
    n = inv.numel()

    def turn(y, weight):
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight
        a, b, rest = y[..., :n], y[..., n:2 * n], y[..., 2 * n:]
        return torch.cat((a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin(), rest), -1)

    q, k = turn(q, w[0]), turn(k, w[1])
    rows = []
    for a, b in bounds:
        seen = ref.seen_mask(b - a, b - a, causal, window, "cuda")
        for h in range(heads):
            z = (scale * q[a:b, h] @ k[a:b, h * kv // heads].T).masked_fill(~seen, -torch.inf)
            rows.append(torch.softmax(z, -1) @ v[a:b, h * kv // heads])
    out = torch.cat([torch.stack(rows[i * heads:(i + 1) * heads], 1) for i in range(len(bounds))])
    out = out.reshape(T, heads * D)
    return (out.detach(), *torch.autograd.grad((out * dout.double()).sum(), (x, *w)))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("window,rot", [(0, None), (20, 16)])
def test_self_attention_module(packed, window, rot):
    """Against float64 autograd.  Roundings to BF16 on the way: q and k after the norm (they move the
    scores by scale * sum |q||k| 2^-8 / sqrt(D), some 2^-8 of p), p, ds, the intermediate gradients and
    the results: five or six of independent sign, the most of each HALF of its entry."""
    say("lm module", packed, window, rot)
    g = torch.Generator().manual_seed(4)
    T, heads, kv, D = 160, 4, 2, 32
    m = lm.SelfAttention(heads, D, kv, rot=rot, window=window, device="cuda")
    with torch.no_grad():
        for p in m.parameters():
            p.add_(_rand(g, D, std=0.2))
    bounds = [(0, 70), (70, 71), (71, 160)] if packed else [(0, T)]
    cu = torch.tensor([0, 70, 71, 160], dtype=torch.int32, device="cuda") if packed else None
    qkv, dout = _rand(g, T, (heads + 2 * kv) * D).requires_grad_(), _rand(g, T, heads * D)
    out = m(qkv, cu=cu)
    out.backward(dout)
    want = _module_reference(m, qkv.detach(), bounds, dout)
    for got, w in zip((out, qkv.grad, m.q_weight.grad, m.k_weight.grad), want):
        _near(got, w, 6 ** 0.5 * HALF)
    if not packed:   # sequences side by side are the same rows
        two = torch.stack((qkv.detach(), qkv.detach())).requires_grad_()
        o2 = m(two)
        assert torch.equal(o2[0], out) and torch.equal(o2[1], out)
        o2.backward(torch.stack((dout, dout)))
        assert torch.equal(two.grad[0], qkv.grad) and torch.equal(two.grad[1], qkv.grad)


def test_module_refuses():
    for bad in (dict(heads=3, dim=32, kv_heads=2), dict(heads=2, dim=20), dict(heads=2, dim=136),
                dict(heads=2, dim=32, rot=34)):
        with pytest.raises(ValueError):
            lm.SelfAttention(**bad)
    m = lm.SelfAttention(2, 16, device="cuda")
    with pytest.raises(ValueError):
        m(torch.zeros(4, 95, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        m(torch.zeros(2, 4, 96, dtype=BF, device="cuda"), cu=torch.zeros(2, dtype=torch.int32, device="cuda"))


def test_captured_step():
    """Forward and backward of the module in one graph, replayed on other rows."""
    say("lm attention graph")
    g = torch.Generator().manual_seed(5)
    m = lm.SelfAttention(4, 64, 2, device="cuda")
    qkv, dout = _rand(g, 300, 8 * 64), _rand(g, 300, 4 * 64)
    params = list(m.parameters())

    def step(x):
        x = x.detach().requires_grad_()
        out = m(x)
        return (out.detach(), *torch.autograd.grad(out, (x, *params), dout))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(qkv)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(qkv)
    for _ in range(4):
        qkv.copy_(_rand(g, *qkv.shape))
        dout.copy_(_rand(g, *dout.shape))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step(qkv)):
            assert torch.equal(a, b)


def test_example_with_attention():
    """The example runs with attention and gives every parameter a finite gradient."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_lm.py")
    spec = importlib.util.spec_from_file_location("train_lm", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    history = ex.train(3, 500, 128, 512, heads=4, document=100)
    assert len(history) == 3 and all(math.isfinite(x) for h in history for x in h)
    model = ex.Model(500, 128, heads=4, document=100)
    ids = torch.randint(0, 500, (512,), device="cuda")
    model(ids, ids).backward()
    for name, p in model.named_parameters():
        assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.abs().max() > 0, name
