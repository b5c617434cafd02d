"""The torch layer of the embedding, head and clipping operators: autograd against
the functional forms and against float64 autograd of the definitions, shapes,
reductions, shared weights, and the example that runs them together."""
import importlib.util
import math
import os

import pytest
import torch

import bit_microscaled_numerics_amd as nv
from bit_microscaled_numerics_amd import lm
from parity import say

pytestmark = pytest.mark.gpu
HALF, U = 2.0 ** -8, 2.0 ** -24


def _data(T=96, V=300, D=64, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, D, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(V, D, generator=g) * 0.2).to(torch.bfloat16).cuda()
    t = torch.randint(0, V, (T,), generator=g)
    t[::7] = -100
    return x, w, t.cuda()


def _reference(x, w, t, row_weight=None):
    """Float64 (token losses, d sum(row_weight * loss) by x and by w)."""
    xr, wr = x.double().cpu().requires_grad_(), w.double().cpu().requires_grad_()
    loss = torch.nn.functional.cross_entropy(xr @ wr.t(), t.cpu().long(), reduction="none",
                                             ignore_index=-100)
    if row_weight is None:
        row_weight = torch.full_like(loss, 1.0 / int((t >= 0).sum()))
    (loss * row_weight.double().cpu()).sum().backward()
    return loss.detach(), xr.grad, wr.grad


def _near(got, ref, rel):
    """Norm-wise: rounding errors of independent sign, each at most `rel` of its entry."""
    assert (got.double().cpu() - ref).norm() <= rel * ref.norm()


@pytest.mark.parametrize("shape", [(96,), (4, 24)])
def test_mean_loss_and_gradients(shape):
    say("lm mean", shape)
    x, w, t = _data()
    x.requires_grad_()
    w.requires_grad_()
    loss = lm.linear_cross_entropy(x.view(*shape, 64), w, t.view(shape))
    assert loss.dtype == torch.float32 and loss.shape == ()
    loss.backward()
    ref, dx, dw = _reference(x.detach(), w.detach(), t)
    n = int((t >= 0).sum())
    assert abs(loss.item() - ref.sum().item() / n) <= 1e-5 * (1 + abs(loss.item()))
    # d rounds to BF16, then the gradient does
    _near(x.grad, dx, 2.5 * HALF)
    _near(w.grad, dw, 2.5 * HALF)
    _, _, fx, fw = nv.linear_ce_grad(x.detach(), w.detach(), t)
    assert torch.equal(x.grad, fx) and torch.equal(w.grad, fw)


def test_incoming_gradient_scales():
    x, w, t = _data()
    x.requires_grad_()
    (lm.linear_cross_entropy(x, w, t) * 3.0).backward()
    _, dx, _ = _reference(x.detach(), w, t)
    _near(x.grad, 3 * dx, 3.5 * HALF)


def test_incoming_gradient_keeps_its_precision():
    """A factor of 1/3 in binary32, not rounded to BF16 first: every entry within a
    binary32 product and half a BF16 step of the exact product; twice, unchanged."""
    x, w, t = _data()
    x.requires_grad_()
    base, = torch.autograd.grad(lm.linear_cross_entropy(x, w, t), x)
    third = torch.tensor(1.0 / 3, device="cuda")
    loss = lm.linear_cross_entropy(x, w, t)
    for _ in range(2):
        got, = torch.autograd.grad(loss, x, third, retain_graph=True)
        ref = base.double() * third.double()
        assert torch.all((got.double() - ref).abs() <= ref.abs() * (U + HALF * (1 + U)))


def test_sum_with_weights_and_tokens_alone():
    x, w, t = _data()
    g = torch.Generator().manual_seed(5)
    weight = torch.rand(96, generator=g).cuda()
    ref, dx, dw = _reference(x, w, t, weight)
    for mode in ("sum", "none"):
        xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
        if mode == "sum":
            loss = lm.linear_cross_entropy(xg, wg, t, weight, reduction="sum")
        else:
            tokens = lm.linear_cross_entropy(xg, wg, t, reduction="none")
            assert tokens.shape == t.shape
            assert torch.all((tokens.double().cpu() - ref).abs() <= 1e-4)
            loss = (tokens * weight).sum()
        assert abs(loss.item() - (ref * weight.double().cpu()).sum().item()) <= 1e-3
        loss.backward()
        _near(xg.grad, dx, 2.5 * HALF)
        _near(wg.grad, dw, 2.5 * HALF)


def test_plain_sum_is_every_weight_one():
    x, w, t = _data()
    x.requires_grad_()
    s = lm.linear_cross_entropy(x, w, t, reduction="sum")
    m = lm.linear_cross_entropy(x, w, t)
    assert abs(s.item() - m.item() * int((t >= 0).sum())) <= 1e-4 * s.item()


def test_without_gradients_nothing_is_kept():
    x, w, t = _data()
    w.requires_grad_()
    with torch.no_grad():
        a = lm.linear_cross_entropy(x, w, t)
    assert not a.requires_grad
    b = lm.linear_cross_entropy(x, w, t)
    assert b.requires_grad and abs(a.item() - b.item()) <= 1e-5 * b.item()


def test_no_target_at_all():
    x, w, t = _data()
    x.requires_grad_()
    loss = lm.linear_cross_entropy(x, w, torch.full_like(t, -100))
    loss.backward()
    assert loss.item() == 0.0 and torch.all(x.grad == 0)


def test_refusals():
    x, w, t = _data()
    with pytest.raises(ValueError, match="reduction"):
        lm.linear_cross_entropy(x, w, t, reduction="max")
    with pytest.raises(ValueError, match="do not match"):
        lm.linear_cross_entropy(x, w, t[:5])
    with pytest.raises(ValueError, match="goes with"):
        lm.linear_cross_entropy(x, w, t, torch.ones(96, device="cuda"))
    with pytest.raises(ValueError, match="row weight"):
        lm.linear_cross_entropy(x, w, t, torch.ones(95, device="cuda"), reduction="sum")
    with pytest.raises(ValueError, match="bf16"):
        lm.linear_cross_entropy(x.float(), w, t)
    with pytest.raises(ValueError, match="columns"):
        lm.linear_cross_entropy(x, w[:, :32].contiguous(), t)
    with pytest.raises(nv.NVFP4Error, match="multiple of 8"):
        lm.linear_cross_entropy(x[:, :60].contiguous(), w[:, :60].contiguous(), t)
    with pytest.raises(ValueError, match="contiguous rows"):
        nv.linear_ce(x.t().contiguous().t(), w, t)
    with pytest.raises(ValueError, match="weight must be"):
        lm.CrossEntropyHead(64, 301, weight=torch.nn.Parameter(w))
    with pytest.raises(ValueError, match="int32 or int64"):
        nv.embed(t.float(), w)
    with pytest.raises(ValueError, match="number of ids"):
        nv.embed_grad(t, x[:5], 300)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_embedding_autograd(dtype):
    g = torch.Generator().manual_seed(2)
    w = torch.randn(50, 40, generator=g).to(dtype).cuda().requires_grad_()
    ids = torch.randint(-1, 51, (6, 11), generator=g).cuda()
    y = lm.EmbeddingFunction.apply(ids, w, 1.5, torch.bfloat16)
    assert y.shape == (6, 11, 40) and y.dtype == torch.bfloat16
    dy = torch.randn(6, 11, 40, generator=g).to(torch.bfloat16).cuda()
    y.backward(dy)
    assert w.grad.dtype == dtype
    assert torch.equal(w.grad, nv.embed_grad(ids.view(-1), dy.view(-1, 40), 50, 1.5, dtype))


def test_embedding_takes_expanded_and_transposed_gradients():
    g = torch.Generator().manual_seed(3)
    w = torch.randn(50, 40, generator=g).cuda().requires_grad_()
    ids = torch.randint(0, 50, (12,), generator=g).cuda()
    count = torch.bincount(ids, minlength=50).float().unsqueeze(1)
    lm.EmbeddingFunction.apply(ids, w, 1.0, torch.float32).sum().backward()   # expanded
    assert torch.equal(w.grad, count.expand(50, 40))
    w.grad = None
    (lm.EmbeddingFunction.apply(ids, w, 1.0, torch.float32).t() * 2.0).contiguous().sum().backward()
    assert torch.equal(w.grad, 2 * count.expand(50, 40))


def test_tied_weight_takes_both_gradients():
    x, w, t = _data(T=32)
    emb = lm.ScaledEmbedding(300, 64, 8.0, "cuda")
    head = lm.CrossEntropyHead(64, 300, "cuda", weight=emb.weight)
    ids = torch.arange(32, device="cuda")
    head(emb(ids), t).backward()
    both = emb.weight.grad.clone()
    y = nv.embed(ids, emb.weight.detach(), 8.0)
    _, _, dy, dw = nv.linear_ce_grad(y, emb.weight.detach(), t)
    de = nv.embed_grad(ids, dy, 300, 8.0)
    assert torch.equal(both, (dw.float() + de.float()).to(torch.bfloat16))


def test_clip_grad_norm():
    g = torch.Generator().manual_seed(4)
    ps = [torch.nn.Parameter(torch.zeros(n, dtype=d, device="cuda"))
          for n, d in ((1000, torch.float32), (37, torch.bfloat16), (5, torch.float32))]
    for p in ps[:2]:
        p.grad = torch.randn(p.shape, generator=g).to(p.dtype).cuda()
    ref = math.sqrt(sum(p.grad.double().square().sum().item() for p in ps[:2]))
    before = [p.grad.clone() for p in ps[:2]]
    norm = lm.clip_grad_norm(ps, 1.0)
    assert abs(norm.item() - ref) <= 1e-6 * ref
    for p, b in zip(ps, before):
        _near(p.grad, b.double().cpu() / (ref + 1e-6), HALF)
    assert lm.clip_grad_norm(ps[2:], 1.0).item() == 0.0


def _example():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "train_lm.py")
    spec = importlib.util.spec_from_file_location("train_lm", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tied", [False, True])
def test_example_learns_and_repeats(tied):
    """The loss starts near log(vocab) (tied: wherever the shared table puts it) and
    falls; a second run gives the same numbers."""
    say("example", tied)
    ex = _example()
    first = ex.train(12, 500, 64, 2048, tied)
    assert all(math.isfinite(v) for step in first for v in step)
    if not tied:
        assert abs(first[0][0] - math.log(500)) < 1.0
    assert first[-1][0] < first[0][0] - 0.1
    assert ex.train(12, 500, 64, 2048, tied) == first


@pytest.mark.parametrize("train", [False, True])
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_loss_of_many_tokens_in_a_graph(train, reduction):
    """The captured loss, replayed on fresh inputs with eager work between, is the eager one."""
    say("lm graph", train, reduction)
    T, V, D = 300007, 40, 8
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    w = torch.randn(V, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    t = torch.randint(-1, V, (T,), generator=torch.Generator().manual_seed(3)).cuda()
    x.requires_grad_(train)
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        lm.linear_cross_entropy(x, w, t, reduction=reduction)
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = lm.linear_cross_entropy(x, w, t, reduction=reduction)
    for seed in range(4):
        g = torch.Generator().manual_seed(10 + seed)
        with torch.no_grad():
            x.copy_(torch.randn(T, D, generator=g))
            t.copy_(torch.randint(-1 - seed, V, (T,), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = loss.item()
        eager = lm.linear_cross_entropy(x, w, t, reduction=reduction).item()
        assert got == eager, seed


@pytest.mark.parametrize("frozen", [False, True])
def test_row_weights_take_a_gradient(frozen):
    """d(sum of weight * loss)/d weight_t is token t's loss, 0 without a target, whether
    x and weight are trained or not."""
    say("lm row weight", frozen)
    x, w, t = _data()
    ref, _, _ = _reference(x, w, t)
    x.requires_grad_(not frozen)
    w.requires_grad_(not frozen)
    rw = torch.rand(96, generator=torch.Generator().manual_seed(6)).cuda().requires_grad_()
    (lm.linear_cross_entropy(x, w, t, rw, reduction="sum") * 2.0).backward()
    assert rw.grad is not None and rw.grad.dtype == torch.float32
    assert torch.all((rw.grad.double().cpu() - 2 * ref).abs() <= 2e-4)
    assert torch.all(rw.grad[t < 0] == 0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_masked_tokens_may_hold_anything(bad):
    """Tokens masked by a weight of 0, or by a choice among the tokens' losses: the loss and
    the gradients are those of the other tokens."""
    say("lm masked", bad)
    x, w, t = _data()
    mask = torch.arange(96, device="cuda") % 5 == 2
    weight = torch.where(mask, 0.0, 0.5)
    zeros = torch.where(mask.unsqueeze(1), torch.zeros_like(x), x)
    ref, dx, dw = _reference(zeros, w, t, weight)
    total = (ref * weight.double().cpu()).sum().item()
    x = torch.where(mask.unsqueeze(1), torch.full_like(x, bad), x)
    for mode in ("weights", "tokens"):
        xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
        if mode == "weights":
            loss = lm.linear_cross_entropy(xg, wg, t, weight, reduction="sum")
        else:
            tokens = lm.linear_cross_entropy(xg, wg, t, reduction="none")
            loss = torch.where(mask, torch.zeros_like(tokens), tokens * 0.5).sum()
        assert abs(loss.item() - total) <= 1e-3
        loss.backward()
        _near(xg.grad, dx, 2.5 * HALF)
        _near(wg.grad, dw, 2.5 * HALF)
        with torch.no_grad():
            assert abs(lm.linear_cross_entropy(x, w, t, weight, reduction="sum").item() - total) <= 1e-3


@pytest.mark.parametrize("lead", [1, 4])
def test_operands_at_any_place_of_a_flat_buffer(lead):
    """A weight (and rows) that start off 16 bytes give what aligned ones give."""
    say("lm flat", lead)
    x, w, t = _data()
    want = lm.linear_cross_entropy(x, w, t)
    wa, xa = w.clone().requires_grad_(), x.clone().requires_grad_()
    lm.linear_cross_entropy(xa, wa, t).backward()
    flat = torch.zeros(w.numel() + x.numel() + 2 * lead, dtype=torch.bfloat16, device="cuda")
    flat[lead:lead + w.numel()].copy_(w.view(-1))
    flat[2 * lead + w.numel():].copy_(x.view(-1))
    wv = flat[lead:lead + w.numel()].view_as(w)
    xv = flat[2 * lead + w.numel():].view_as(x)
    assert torch.equal(lm.linear_cross_entropy(xv, wv, t), want)
    tokens = lm.linear_cross_entropy(xv, wv, t, reduction="none")
    assert torch.equal(tokens, lm.linear_cross_entropy(x, w, t, reduction="none"))
    wp, xp = wv.detach().requires_grad_(), xv.detach().requires_grad_()
    assert wp.data_ptr() % 16 != 0
    lm.linear_cross_entropy(xp, wp, t).backward()
    assert torch.equal(wp.grad, wa.grad) and torch.equal(xp.grad, xa.grad)


@pytest.mark.parametrize("train_x,train_w", [(True, False), (False, True)])
def test_one_side_frozen(train_x, train_w):
    x, w, t = _data()
    _, _, dx, dw = nv.linear_ce_grad(x, w, t)
    x.requires_grad_(train_x)
    w.requires_grad_(train_w)
    lm.linear_cross_entropy(x, w, t).backward()
    assert torch.equal(x.grad, dx) if train_x else x.grad is None
    assert torch.equal(w.grad, dw) if train_w else w.grad is None


def test_clip_of_one_parameter_and_of_a_transposed_one():
    p = torch.nn.Parameter(torch.zeros(6, 40, device="cuda").t())
    g = torch.Generator().manual_seed(8)
    (p * torch.randn(40, 6, generator=g).cuda()).sum().backward()
    assert not p.grad.is_contiguous()
    before = p.grad.double().cpu()
    assert abs(lm.clip_grad_norm(p, 1.0).item() - before.norm().item()) <= 1e-6 * before.norm()
    _near(p.grad, before / (before.norm() + 1e-6), 4 * U)
