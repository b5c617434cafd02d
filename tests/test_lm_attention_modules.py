"""The torch layer of attention on the CPU, with the library's calls replaced by their
definitions: what is handed on, what is copied, what is differentiable."""
import pytest
import torch

from bit_microscaled_numerics_amd import lm


def _attend(q, k, v, scale, causal, window, cu_q=None, cu_k=None):
    G = q.shape[-2] // k.shape[-2]
    q, k, v = (x.float().transpose(-2, -3) for x in (q, k, v))
    k, v = (x.repeat_interleave(G, -3) for x in (k, v))
    z = (q.shape[-1] ** -0.5 if scale is None else scale) * q @ k.transpose(-1, -2)
    if causal:
        z = z.masked_fill(~torch.ones(z.shape[-2:], dtype=torch.bool).tril(z.shape[-1] - z.shape[-2]), -torch.inf)
    lse = torch.logsumexp(z, -1)
    return (torch.exp(z - lse.unsqueeze(-1)) @ v).transpose(-2, -3), lse.transpose(-1, -2)


@pytest.fixture
def calls(monkeypatch):
    log = []

    def forward(q, k, v, scale, causal, window, cu_q=None, cu_k=None):
        log.append((q, k, v))
        out, lse = _attend(q, k, v, scale, causal, window)
        return out.to(q.dtype).contiguous(), lse.contiguous()

    def grad(dout, q, k, v, out, lse, scale, causal, window, cu_q=None, cu_k=None, grads=None):
        log.append((dout,))
        with torch.enable_grad():
            leaves = [x.detach().float().requires_grad_() for x in (q, k, v)]
            o, _ = _attend(*leaves, scale, causal, window)
            res = torch.autograd.grad((o * dout.float()).sum(), leaves)
        return tuple(r.to(x.dtype) for r, x in zip(res, (q, k, v)))

    monkeypatch.setattr(lm, "attention_forward", forward)
    monkeypatch.setattr(lm, "attention_grad", grad)
    return log


def _rand(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)


@pytest.mark.parametrize("train", [(True, True, True), (True, False, False), (False, False, True)])
def test_gradients_go_where_they_are_asked_for(calls, train):
    args = [_rand(2, 9, H, 16).requires_grad_(t) for H, t in zip((4, 2, 2), train)]
    out = lm.attention(*args, causal=True)
    out.sum().backward()   # an expanded gradient
    for x, t in zip(args, train):
        assert (x.grad is not None) == t
        assert not t or x.grad.shape == x.shape
    assert calls[-1][0].stride(-1) == 1 and calls[-1][0].stride(0) > 0


def test_operands_off_16_bytes_are_copied(calls):
    flat = torch.zeros(9 * 4 * 16 + 4, dtype=torch.bfloat16)
    x = flat[4:].view(9, 4, 16)
    assert x.data_ptr() % 16
    lm.attention(x, x, x)
    assert all(y.data_ptr() % 16 == 0 for y in calls[0])
    wide = torch.zeros(9, 4, 20, dtype=torch.bfloat16)[..., :16]   # a stride of 20
    lm.attention(wide, wide, wide)
    assert all(y.stride(1) == 16 for y in calls[1])
    heads_first = torch.zeros(4, 9, 16, dtype=torch.bfloat16).transpose(0, 1)
    lm.attention(heads_first, heads_first, heads_first)
    assert all(y.data_ptr() == heads_first.data_ptr() for y in calls[2])   # taken as it lies


def test_shapes_that_do_not_match():
    with pytest.raises(ValueError):
        lm.qk_norm_rope(_rand(3, 2, 16), _rand(4, 2, 16))
    m = lm.SelfAttention(4, 16, 2)
    for bad in (_rand(5, 100), _rand(128), _rand(1, 1, 5, 128)):
        with pytest.raises(ValueError):
            m(bad)
    with pytest.raises(ValueError):
        m(_rand(1, 5, 128), cu=torch.zeros(2, dtype=torch.int32))
