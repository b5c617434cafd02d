"""The torch layer of SelfAttention on the CPU, with the library's calls replaced: casts of the module, calls
without tokens, rows that overlap."""
import copy

import pytest
import torch

from bit_microscaled_numerics_amd import lm

BF = torch.bfloat16


def _fresh(**kw):
    return lm.SelfAttention(4, 16, 2, base=5e5, **kw)


@pytest.mark.parametrize("change", [
    lambda m: m.to(BF), lambda m: m.bfloat16(), lambda m: m.half(), lambda m: m.double(), lambda m: m.bfloat16().float(),
    lambda m: m.half().to(torch.float32), lambda m: torch.nn.Sequential(m).to(BF)[0], lambda m: copy.deepcopy(m).to(BF),
    lambda m: m.to("cpu", BF)])
@pytest.mark.parametrize("rot", [None, 6, 0])
def test_casts_leave_the_frequencies(change, rot):
    want = _fresh(rot=rot).inv_freq
    m = change(_fresh(rot=rot))
    assert m.inv_freq.dtype == torch.float32 and torch.equal(m.inv_freq, want)
    assert "inv_freq" not in m.state_dict() and "inv_freq" in dict(m.named_buffers())


def test_casts_cast_the_weights():
    m = _fresh()
    assert m.q_weight.dtype == BF and m.float().q_weight.dtype == torch.float32 and m.to(BF).k_weight.dtype == BF


def test_module_made_without_memory():
    """Made on the meta device and given memory, the buffer included, which nothing would fill."""
    m = _fresh(device="meta")
    assert m.inv_freq.is_meta and m.inv_freq.dtype == torch.float32
    m.to_empty(device="cpu")
    assert torch.equal(m.inv_freq, _fresh().inv_freq)
    with torch.device("meta"):
        m = _fresh()
    assert m.inv_freq.is_meta and m.to(BF).inv_freq.dtype == torch.float32


def test_a_change_of_nothing_keeps_the_buffer():
    """A captured graph reads it where it lies."""
    m = _fresh()
    at = m.inv_freq.data_ptr()
    assert m.to(torch.float32).inv_freq.data_ptr() == at and m.to("cpu").inv_freq.data_ptr() == at


def test_frequencies_put_in_are_kept():
    m = _fresh()
    own = torch.rand(8)
    m.inv_freq = own.clone()
    for change in (lambda: m.to(BF), m.half, m.float, lambda: m.to_empty(device="cpu")):
        change()
        assert m.inv_freq.dtype == torch.float32 and torch.equal(m.inv_freq, own)


@pytest.fixture
def calls(monkeypatch):
    """The module's calls of the library, with results of the right shapes."""
    log = []

    def rope(q, k, *rest, **kw):
        assert q.shape[0] == k.shape[0] and (rest[2] is None or rest[2].numel() == q.shape[0])
        return (q.clone(memory_format=torch.contiguous_format), k.clone(memory_format=torch.contiguous_format))

    def rope_grad(dq, dk, q, k, q_weight=None, k_weight=None, *rest, out=None, **kw):
        dw = [None if w is None else torch.zeros_like(w) for w in (q_weight, k_weight)]
        return (*((dq, dk) if out is None else out), *dw)

    def forward(q, k, v, *rest, **kw):
        log.append((q, k, v))
        return torch.zeros(q.shape, dtype=q.dtype), torch.zeros(q.shape[:-1])

    def grad(dout, q, k, v, out, lse, *rest, grads=None, **kw):
        assert dout.shape == q.shape
        for x, like in zip(grads, (q, k, v)):
            assert x.shape == like.shape
            x.zero_()
        return grads

    for name, fn in (("qk_norm_rope_forward", rope), ("qk_norm_rope_grad", rope_grad),
                     ("attention_forward", forward), ("attention_grad", grad)):
        monkeypatch.setattr(lm, name, fn)
    return log


@pytest.mark.parametrize("shape", [(0,), (2, 0), (0, 3), (0, 0)])
@pytest.mark.parametrize("norm", [True, False])
def test_no_tokens(calls, shape, norm):
    m = _fresh(norm=norm)
    x = torch.zeros(*shape, 128, dtype=BF, requires_grad=True)
    for kw in (dict(), dict(positions=torch.zeros((), dtype=torch.int64))):
        out = m(x, **kw)
        assert out.shape == (*shape, 64)
        out.backward(torch.zeros_like(out))
        assert x.grad.shape == x.shape and all(not p.grad.any() for p in m.parameters())
    if len(shape) == 1:
        for cu in ([0], [0, 0], [0, 0, 0]):
            assert m(x, cu=torch.tensor(cu, dtype=torch.int32)).shape == (0, 64)


def test_rows_that_overlap_are_copied(calls):
    """Windows that slide over one row of tokens share its rows; attention takes rows apart."""
    tokens = torch.zeros(10, 128, dtype=BF, requires_grad=True)
    windows = tokens.unfold(0, 4, 2).transpose(1, 2)   # [4][4][128], every second token in two of them
    assert windows.stride() == (256, 128, 1)
    m = _fresh()
    out = m(windows)
    out.backward(torch.zeros_like(out))
    assert tokens.grad.shape == tokens.shape
    m(windows.expand(4, 4, 128)[:1].expand(3, 4, 128))
    for q, k, v in calls:
        assert v.stride() == (4 * 128, 128, 16, 1)
    apart = torch.zeros(4, 3, 128, dtype=BF).transpose(0, 1)
    m(apart)
    assert calls[-1][2].stride() == (128, 3 * 128, 16, 1)   # taken as it lies
