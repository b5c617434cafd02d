"""The torch layer of the head and its loss on the CPU, with the library's calls replaced
by their definitions: what is differentiable, what is handed on, what is refused."""
import pytest
import torch

from bit_microscaled_numerics_amd import lm


def _ce(h, w, t):
    """nv.linear_ce's contract in binary32: (loss, lse)."""
    z = h.float() @ w.float().t()
    live = (t >= 0) & (t < w.shape[0])
    at = t.clamp(0, w.shape[0] - 1).long().unsqueeze(1)
    lse = torch.logsumexp(z, 1)
    return torch.where(live, lse - z.gather(1, at).squeeze(1), torch.zeros_like(lse)), lse


def _ce_grad(h, w, t, row_weight=None, piece_tokens=0):
    """nv.linear_ce_grad's contract: (loss, lse, dh, dw)."""
    live = (t >= 0) & (t < w.shape[0])
    if row_weight is None:
        row_weight = torch.full((h.shape[0],), 1.0 / max(1, int(live.sum())))
    with torch.enable_grad():
        hr, wr = h.detach().float().requires_grad_(), w.detach().float().requires_grad_()
        loss, lse = _ce(hr, wr, t)
        dh, dw = torch.autograd.grad((loss * row_weight.detach()).sum(), (hr, wr))
    return loss.detach(), lse.detach(), dh.to(h.dtype), dw.to(w.dtype)


@pytest.fixture
def calls(monkeypatch):
    """The definitions in place of the library; collects what they are given."""
    log = {"operands": [], "scaled": []}

    def ce(h, w, t):
        log["operands"].append((h, w))
        return _ce(h, w, t)

    def ce_grad(h, w, t, row_weight=None, piece_tokens=0):
        log["operands"].append((h, w))
        return _ce_grad(h, w, t, row_weight, piece_tokens)

    def scale(grads, factor):
        log["scaled"].append(len(grads))
        return [(g.float() * factor).to(g.dtype) for g in grads]

    monkeypatch.setattr(lm, "linear_ce", ce)
    monkeypatch.setattr(lm, "linear_ce_grad", ce_grad)
    monkeypatch.setattr(lm, "scale_grads", scale)
    return log


def _data(T=24, V=30, D=16):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(T, D, generator=g).to(torch.bfloat16)
    w = (torch.randn(V, D, generator=g) * 0.2).to(torch.bfloat16)
    t = torch.randint(0, V, (T,), generator=g)
    t[::5] = -100
    return x, w, t


@pytest.mark.parametrize("shape", [(24,), (4, 6)])
@pytest.mark.parametrize("train_x,train_w", [(True, True), (True, False), (False, True),
                                             (False, False)])
def test_row_weights_take_a_gradient(calls, shape, train_x, train_w):
    """d(sum of weight * loss)/d weight_t = loss_t whichever of x and weight is trained."""
    x, w, t = _data()
    loss, _ = _ce(x, w, t)
    x.requires_grad_(train_x)
    w.requires_grad_(train_w)
    rw = torch.rand(24, generator=torch.Generator().manual_seed(1)).view(shape).requires_grad_()
    out = lm.linear_cross_entropy(x.view(*shape, 16), w, t.view(shape), rw, reduction="sum")
    (out * 3.0).backward()
    assert rw.grad.shape == shape
    assert torch.allclose(rw.grad.reshape(-1), 3 * loss, rtol=1e-6, atol=0)
    assert torch.all(rw.grad.reshape(-1)[t < 0] == 0)
    # a weight formed from parameters trains them
    a = torch.tensor(0.5, requires_grad=True)
    lm.linear_cross_entropy(x.view(*shape, 16), w, t.view(shape), torch.exp(a).expand(shape),
                            reduction="sum").backward()
    want = loss.sum().item() * torch.exp(torch.tensor(0.5)).item()
    assert abs(a.grad.item() - want) <= 1e-5 * want


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("train", [False, True])
def test_losses_of_weight_zero_do_not_count(calls, bad, train):
    """A masked token's loss that is not finite stays out of the sum; a finite one still
    has its derivative by the weight."""
    x, w, t = _data()
    loss, _ = _ce(x, w, t)
    weight = torch.full((24,), 0.5)
    weight[7] = weight[8] = 0.0
    want = (loss * weight).sum().item()
    x[7] = bad
    x.requires_grad_(train)
    weight.requires_grad_()
    out = lm.linear_cross_entropy(x, w, t, weight, reduction="sum")
    assert abs(out.item() - want) <= 1e-5 * want
    out.backward()
    keep = torch.arange(24) != 7
    assert torch.allclose(weight.grad[keep], loss[keep], rtol=1e-6, atol=0)


@pytest.mark.parametrize("lead", [0, 1, 4, 8])
@pytest.mark.parametrize("mode", ["train", "none", "score"])
def test_operands_at_any_place_of_a_flat_buffer(calls, lead, mode):
    """What the products are given starts on 16 bytes; gradients reach the pieces."""
    x, w, t = _data()
    flat = torch.zeros(2 * lead + w.numel() + x.numel(), dtype=torch.bfloat16)
    wv = flat[lead:lead + w.numel()].view_as(w).copy_(w)
    xv = flat[2 * lead + w.numel():].view_as(x).copy_(x)
    if mode == "score":
        assert lm.linear_cross_entropy(xv, wv, t) == lm.linear_cross_entropy(x, w, t)
    else:
        wv, xv = wv.detach().requires_grad_(), xv.detach().requires_grad_()
        w.requires_grad_()
        x.requires_grad_()
        kw = dict(reduction="none") if mode == "none" else {}
        lm.linear_cross_entropy(xv, wv, t, **kw).sum().backward()
        lm.linear_cross_entropy(x, w, t, **kw).sum().backward()
        assert torch.equal(xv.grad, x.grad) and torch.equal(wv.grad, w.grad)
    assert all(o.data_ptr() % 16 == 0 for pair in calls["operands"] for o in pair)
    # aligned operands are handed on as they are
    if mode == "score" and lead in (0, 8):
        assert calls["operands"][0][1].data_ptr() == wv.data_ptr()


def test_rows_off_their_pitch_are_copied(calls):
    x, w, t = _data()
    wide = torch.zeros(30, 19, dtype=torch.bfloat16)
    wide[:, :16] = w
    assert lm.linear_cross_entropy(x, wide[:, :16], t) == lm.linear_cross_entropy(x, w, t)
    assert calls["operands"][0][1].stride(0) == 16


def test_float32_table_cannot_be_shared_with_a_head():
    """Refused where the model is put together, not by its first loss."""
    table = lm.ScaledEmbedding(30, 16, dtype=torch.float32)
    with pytest.raises(ValueError, match="bf16"):
        lm.CrossEntropyHead(16, 30, weight=table.weight)
    tied = lm.ScaledEmbedding(30, 16)
    assert lm.CrossEntropyHead(16, 30, weight=tied.weight).weight is tied.weight


@pytest.mark.parametrize("train_x,train_w", [(True, True), (True, False), (False, True)])
def test_gradients_nobody_asks_for_are_not_kept(calls, train_x, train_w):
    x, w, t = _data()
    _, _, dx, dw = _ce_grad(x, w, t)
    x.requires_grad_(train_x)
    w.requires_grad_(train_w)
    loss = lm.linear_cross_entropy(x, w, t)
    kept = [s for s in loss.grad_fn.saved_tensors if s is not None]
    assert [tuple(s.shape) for s in kept] == [(24, 16)] * train_x + [(30, 16)] * train_w
    loss.backward()
    assert calls["scaled"] == [train_x + train_w]
    assert torch.equal(x.grad, dx) if train_x else x.grad is None
    assert torch.equal(w.grad, dw) if train_w else w.grad is None


def _clip(grads, max_norm, partials=None):
    """nv.clip_grads's contract in place: what is not contiguous is refused."""
    if not all(g.is_contiguous() for g in grads):
        raise ValueError("gradients must be contiguous")
    norm = sum(g.double().square().sum() for g in grads).sqrt()
    for g in grads:
        g.mul_(min(1.0, max_norm / (norm.item() + 1e-6)))
    return norm.float().reshape(1)


def test_one_parameter_is_clipped(monkeypatch):
    """A parameter by itself, not an iterable of its rows (which have no gradients)."""
    monkeypatch.setattr(lm, "clip_grads", _clip)
    p = torch.nn.Parameter(torch.zeros(4, 4))
    p.grad = torch.ones(4, 4)
    assert lm.clip_grad_norm(p, 1.0).item() == 4.0
    assert torch.allclose(p.grad, torch.full((4, 4), 0.25))


def test_gradients_in_another_order_of_memory_are_clipped(monkeypatch):
    """A transposed (or channels-last) parameter's gradient has its strides; gaps are refused."""
    monkeypatch.setattr(lm, "clip_grads", _clip)
    ps = [torch.nn.Parameter(torch.zeros(4, 6).t()),
          torch.nn.Parameter(torch.zeros(2, 3, 5, 4).to(memory_format=torch.channels_last)),
          torch.nn.Parameter(torch.zeros(3, 1, 2).transpose(0, 2)), torch.nn.Parameter(torch.zeros(5))]
    g = torch.Generator().manual_seed(0)
    for p in ps:
        p.grad = torch.empty_like(p).copy_(torch.randn(p.shape, generator=g))
    before = [p.grad.clone() for p in ps]
    assert not ps[0].grad.is_contiguous() and not ps[1].grad.is_contiguous()
    norm = lm.clip_grad_norm(ps, 1.0).item()
    want = sum(b.double().square().sum() for b in before).sqrt().item()
    assert abs(norm - want) <= 1e-6 * want
    for p, b in zip(ps, before):
        assert p.grad.stride() == b.stride()
        assert torch.allclose(p.grad, b / want, rtol=1e-5, atol=1e-7)
    p = torch.nn.Parameter(torch.zeros(4, 6))
    p.grad = torch.ones(4, 12)[:, ::2]
    with pytest.raises(ValueError, match="contiguous"):
        lm.clip_grad_norm([p], 1.0)
