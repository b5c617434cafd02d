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
