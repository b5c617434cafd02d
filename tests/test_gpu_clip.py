"""Global gradient norm and clipping against 64-bit references.

Tolerances: the norm is a binary64 sum rounded to binary32 once (2^-24; the
binary64 sum of n squares is within n * 2^-53).  An output is the gradient
times a binary32 factor (2^-24 and the norm's own 2^-24 do not matter: the
factor is formed in binary64), one product rounding, and half a step of its
type; below the normal range a half step is a fixed 2^-150 (binary32) or 2^-134
(BF16)."""
import math

import pytest
import torch

import bit_microscaled_numerics_amd as nv
from parity import say

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U32 = 2.0 ** -24
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
BF, F = torch.bfloat16, torch.float32


def _ref(grads, max_norm):
    norm = math.sqrt(math.fsum(g.double().square().sum().item() for g in grads))
    coef = min(1.0, max_norm / (norm + 1e-6))
    return norm, [g.double() * coef for g in grads]


def _check(norm, outs, grads, max_norm):
    rn, ro = _ref(grads, max_norm)
    assert norm.shape == (1,) and norm.dtype == F
    assert abs(norm.item() - rn) <= rn * (U32 + 1e-9)
    for o, r in zip(outs, ro):
        tol = r.abs() * (3 * U32 + HALF[o.dtype] * (1 + 3 * U32)) + LEAST[F] + LEAST[o.dtype]
        assert torch.all((o.cpu().double() - r).abs() <= tol)


def _grads(seed, sizes, dtypes, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(dtypes[i % len(dtypes)]) for i, n in enumerate(sizes)]


CHUNK = 32768   # bytes of a workgroup's chunk
SIZES = {
    "one": [1], "few": [7, 8, 9, 0, 1], "empty": [0, 0],
    "chunk": [CHUNK // 4, CHUNK // 2, CHUNK // 4 + 1, CHUNK // 2 - 1],
    "many": [3 + 5 * i for i in range(300)],                      # several batches of 96
    "past_grid": [CHUNK // 4 * 700 + 13, 5, CHUNK // 2 * 400 + 1],   # chunks past the 512 workgroups
}


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtypes", [(BF,), (F,), (F, BF)], ids=["bf16", "f32", "mixed"])
@pytest.mark.parametrize("max_norm", [1.0, 1e6])
def test_in_place(sizes, dtypes, max_norm):
    say("clip", sizes, dtypes, max_norm)
    grads = _grads(1, SIZES[sizes], dtypes)
    dev = [g.cuda() for g in grads]
    norm = nv.clip_grads(dev, max_norm)
    _check(norm, dev, grads, max_norm)
    if max_norm == 1e6:
        assert all(torch.equal(d.cpu(), g) for d, g in zip(dev, grads))


@pytest.mark.parametrize("dt,ot", [(BF, F), (F, BF), (F, F), (BF, BF)])
@pytest.mark.parametrize("max_norm", [0.5, float("inf"), 0.0])
def test_into_outputs(dt, ot, max_norm):
    say("clip out", dt, ot, max_norm)
    grads = _grads(2, [1000, 3, 40000], (dt,))
    dev = [g.cuda() for g in grads]
    outs = [torch.full(g.shape, 9.0, dtype=ot, device="cuda") for g in grads]
    norm = nv.clip_grads(dev, max_norm, out=outs)
    _check(norm, outs, grads, max_norm)
    assert all(torch.equal(d.cpu(), g) for d, g in zip(dev, grads))


@pytest.mark.parametrize("dt", [BF, F])
def test_pieces_of_a_flat_buffer(dt):
    """Tensors that start at any element, with their neighbours watched."""
    sizes = [1, 31, 4097, 2, 70001, 5]
    say("clip flat", dt)
    flat = _grads(3, [sum(sizes) + 2], (dt,))[0]
    dev = flat.cuda()
    views = list(dev[1:-1].split(sizes))
    norm = nv.clip_grads(views, 1.0)
    _check(norm, views, list(flat[1:-1].split(sizes)), 1.0)
    assert dev[0].item() == flat[0].item() and dev[-1].item() == flat[-1].item()


@pytest.mark.parametrize("scale", [1e-30, 1e25])
def test_squares_beyond_binary32(scale):
    grads = _grads(4, [5000], (F,), std=scale)
    dev = [g.cuda() for g in grads]
    norm = nv.clip_grads(dev, scale)
    _check(norm, dev, grads, scale)


def test_nonfinite_norms():
    a = torch.ones(100, device="cuda")
    b = torch.ones(50, device="cuda", dtype=BF)
    b[3] = float("inf")
    norm = nv.clip_grads([a, b], 1.0)
    assert math.isinf(norm.item()) and torch.all(a == 0)
    assert torch.isnan(b[3]) and torch.all(b[:3] == 0)
    a = torch.ones(100, device="cuda")
    b = torch.ones(50, device="cuda", dtype=BF)
    a[7] = float("nan")
    norm = nv.clip_grads([a, b], 1.0)
    assert math.isnan(norm.item()) and torch.isnan(a).all() and torch.isnan(b).all()


def test_partials_add_up_over_shards():
    """Two shards' partial sums added word by word clip as one list does."""
    grads = _grads(5, [4000, 123, 9], (F, BF))
    dev = [g.cuda() for g in grads]
    total = nv.grad_sumsq(dev[:1]) + nv.grad_sumsq(dev[1:])
    assert total.dtype == torch.float64 and total.numel() == nv.NVFP4_SUMSQ_WORDS
    norm = nv.clip_grads(dev, 1.0, partials=total)
    _check(norm, dev, grads, 1.0)


def test_same_bits_every_time_and_in_a_graph():
    grads = _grads(6, [100003, 17, 5], (F, BF))
    dev = [g.cuda() for g in grads]
    outs = [torch.empty_like(d) for d in dev]
    partials = torch.empty(nv.NVFP4_SUMSQ_WORDS, dtype=torch.float64, device="cuda")
    norm = torch.empty(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_grad_sumsq(dev, partials)
        nv.nvfp4_grad_clip(dev, outs, partials, 1.0, norm)
    for k in range(3):
        fresh = _grads(7 + k, [100003, 17, 5], (F, BF))
        for d, f in zip(dev, fresh):
            d.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        _check(norm, outs, fresh, 1.0)
        eager = [torch.empty_like(d) for d in dev]
        assert torch.equal(nv.clip_grads(dev, 1.0, out=eager), norm)
        assert all(torch.equal(a, b) for a, b in zip(eager, outs))


def test_on_another_stream():
    grads = _grads(8, [50000], (F,))
    dev = [g.cuda() for g in grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        norm = nv.clip_grads(dev, 1.0)
    side.synchronize()
    _check(norm, dev, grads, 1.0)


@pytest.mark.parametrize("dt,ot", [(BF, BF), (F, BF), (BF, F), (F, F)])
@pytest.mark.parametrize("factor", [1.0, 1.0 / 3, -2.5, 0.0])
def test_scale(dt, ot, factor):
    """out = in * factor, the factor in binary32 (not rounded to the gradients' type)."""
    say("scale", dt, ot, factor)
    grads = _grads(9, [1003, 0, 7, 40000], (dt,))
    dev = [g.cuda() for g in grads]
    outs = [torch.full(g.shape, 9.0, dtype=ot, device="cuda") for g in grads]
    f = torch.tensor([factor], dtype=torch.float32, device="cuda")
    nv.nvfp4_grad_scale(dev, outs, f)
    for o, g in zip(outs, grads):
        r = g.double() * f.double().item()
        assert torch.all((o.cpu().double() - r).abs() <= r.abs() * (U32 + HALF[ot] * (1 + U32)))
    if dt == ot:
        new = nv.scale_grads(dev, f)
        assert all(torch.equal(a, b) for a, b in zip(new, outs))
        nv.nvfp4_grad_scale(dev, dev, f)
        assert all(torch.equal(a, b) for a, b in zip(dev, outs))


def test_lists_that_are_read_once():
    """Generators: every gradient counts."""
    grads = _grads(11, [1000, 7, 31, 4], (F, BF))
    dev = [g.cuda() for g in grads]
    outs = [torch.empty_like(g) for g in dev]
    partials = torch.empty(nv.NVFP4_SUMSQ_WORDS, dtype=torch.float64, device="cuda")
    norm = torch.empty(1, device="cuda")
    nv.nvfp4_grad_sumsq((g for g in dev), partials)
    nv.nvfp4_grad_clip((g for g in dev), (o for o in outs), partials, 1.0, norm)
    _check(norm, outs, grads, 1.0)


def test_norm_and_factor_have_to_be_on_the_gpu():
    dev = [torch.ones(5, device="cuda")]
    partials = nv.grad_sumsq(dev)
    for bad in (torch.zeros(1), torch.zeros(1, dtype=BF, device="cuda"), torch.zeros(2, device="cuda")):
        with pytest.raises(ValueError, match="norm_out"):
            nv.nvfp4_grad_clip(dev, dev, partials, 1.0, bad)
        with pytest.raises(ValueError, match="factor"):
            nv.nvfp4_grad_scale(dev, dev, bad)
    nv.nvfp4_grad_clip(dev, dev, partials, 100.0, None)   # the norm is not wanted
    assert torch.all(dev[0] == 1)


def test_gradients_without_a_dimension():
    """0-dimensional gradients (a scalar parameter's) scale, clip and count like others."""
    grads = [torch.tensor(3.0), torch.tensor([4.0, 0.0])]
    dev = [g.cuda() for g in grads]
    new = nv.scale_grads(dev, torch.tensor([0.5], device="cuda"))
    assert [g.shape for g in new] == [(), (2,)]
    assert new[0].item() == 1.5 and new[1].tolist() == [2.0, 0.0]
    norm = nv.clip_grads(dev, 1.0)
    _check(norm, dev, grads, 1.0)
