"""Embedding lookup and its gradient against 64-bit references.

Tolerances, per entry: the lookup rounds a binary32 product once (2^-24) and
the output once (half a step of its type).  The gradient adds n terms in
binary32, at most n roundings of 2^-24 relative to the sum of magnitudes, one
for the scale, and the output's half step."""
import numpy as np
import pytest
import torch

import bit_microscaled_numerics_amd as nv
from parity import say

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U32 = 2.0 ** -24


def _rand(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _ids(g, n, V, kind, dtype):
    if kind == "same":
        t = torch.full((n,), V // 2)
    elif kind == "zipf":
        t = torch.exp(torch.rand(n, generator=g) * np.log(V)).long().clamp(1, V) - 1
    elif kind == "outside":   # a third of the tokens carry no word
        t = torch.randint(0, V, (n,), generator=g)
        r = torch.rand(n, generator=g)
        t = torch.where(r < 0.2, torch.full_like(t, -1), torch.where(r < 0.33, t + V, t))
    else:
        t = torch.randint(0, V, (n,), generator=g)
    return t.to(dtype)


def _strided(x, pad, lead):
    """x on the GPU with `pad` extra columns, starting `lead` elements into its buffer."""
    n, d = x.shape
    buf = torch.full((n * (d + pad) + lead,), 7.0, dtype=x.dtype, device="cuda")
    v = buf[lead:].view(n, d + pad)[:, :d]
    v.copy_(x)
    return v


@pytest.mark.parametrize("n", [0, 1, 3, 64, 2047, 2500])
@pytest.mark.parametrize("D", [1, 7, 8, 64, 511, 512, 2056, 2600])
@pytest.mark.parametrize("wt,ot", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16),
                                   (torch.bfloat16, torch.float32), (torch.float32, torch.float32)])
def test_lookup(n, D, wt, ot):
    say("embed", n, D, wt, ot)
    g = torch.Generator().manual_seed(n * 1000 + D)
    V, scale = 37, 2.7
    w = _rand(g, V, D, dtype=wt)
    ids = _ids(g, n, V, "outside", torch.int64 if D % 2 else torch.int32)
    out = nv.embed(ids.cuda(), w.cuda(), scale, dtype=ot).cpu().double()
    live = ((ids >= 0) & (ids < V)).unsqueeze(1)
    ref = w.double()[ids.long().clamp(0, V - 1)] * float(np.float32(scale)) * live
    assert out.shape == ref.shape
    assert torch.all((out - ref).abs() <= ref.abs() * (U32 + HALF[ot] * (1 + U32)))


def test_lookup_strides_and_c_entry():
    g = torch.Generator().manual_seed(3)
    w = _rand(g, 50, 100, dtype=torch.bfloat16)
    ids = _ids(g, 77, 50, "uniform", torch.int32).cuda()
    for pad, lead in [(1, 1), (3, 0), (28, 5)]:
        say("embed strides", pad, lead)
        out = torch.full((77, 100 + pad), -3.0, dtype=torch.float32, device="cuda")
        nv.nvfp4_embed(ids, _strided(w, pad, lead), 0.5, out[:, :100])
        assert torch.equal(out[:, :100].cpu(), w.float()[ids.cpu().long()] * 0.5)
        assert torch.all(out[:, 100:] == -3.0)


def test_nonfinite_words_stay_with_their_tokens():
    w = torch.zeros(4, 16, dtype=torch.float32)
    w[1], w[2] = float("inf"), float("nan")
    ids = torch.tensor([0, 1, 2, -1, 3], device="cuda")
    out = nv.embed(ids, w.cuda(), 2.0, dtype=torch.bfloat16).cpu()
    assert torch.isinf(out[1]).all() and torch.isnan(out[2]).all()
    assert torch.all(out[[0, 3, 4]] == 0)


def _ref_grad(ids, dy, V, scale):
    live = (ids >= 0) & (ids < V)
    at = ids[live].long()
    s = float(np.float32(scale))
    d = dy.double()[live]
    ref = torch.zeros(V, dy.shape[1], dtype=torch.float64).index_add_(0, at, d) * s
    mag = torch.zeros(V, dy.shape[1], dtype=torch.float64).index_add_(0, at, d.abs()) * abs(s)
    count = torch.bincount(at, minlength=V).double().unsqueeze(1)
    return ref, mag, count


def _check_grad(got, ids, dy, V, scale, base=None):
    ref, mag, count = _ref_grad(ids, dy, V, scale)
    if base is not None:
        ref, mag, count = ref + base.double(), mag + base.double().abs(), count + 1
    tol = (count + 1) * U32 * mag * 1.01 + HALF[got.dtype] * (ref.abs() + (count + 1) * U32 * mag)
    err = (got.cpu().double() - ref).abs()
    bad = torch.nonzero(~(err <= tol))
    assert bad.numel() == 0, (len(bad), bad[0].tolist(), err.max().item())


# sizes around the sort's steps (1024, 4096, 8192, 16384 tokens), the window of
# 64 and tiles of 4096 of the larger sort
@pytest.mark.parametrize("n", [0, 1, 63, 64, 65, 1024, 1025, 4097, 8193, 16384, 16385, 20481])
@pytest.mark.parametrize("kind", ["uniform", "same", "zipf", "outside"])
@pytest.mark.parametrize("V,D", [(1, 8), (511, 9), (512, 64), (5003, 40)])
def test_gradient(n, kind, V, D):
    say("embed_grad", n, kind, V, D)
    g = torch.Generator().manual_seed(n + V)
    yt = torch.bfloat16 if (n + D) % 2 else torch.float32
    wt = torch.bfloat16 if V % 2 else torch.float32
    ids = _ids(g, n, V, kind, torch.int32 if n % 2 else torch.int64)
    dy = _rand(g, n, D, dtype=yt)
    got = nv.embed_grad(ids.cuda(), dy.cuda(), V, 1.7, dtype=wt)
    _check_grad(got, ids, dy, V, 1.7)


@pytest.mark.parametrize("n", [32767, 32768, 32769, 36865, 70000])
@pytest.mark.parametrize("kind", ["uniform", "same", "zipf", "outside"])
def test_gradient_of_many_tokens(n, kind):
    """Both sides of the largest merged sort (8 tiles of 4096)."""
    say("embed_grad many", n, kind)
    g = torch.Generator().manual_seed(n)
    V, D = 997, 24
    ids = _ids(g, n, V, kind, torch.int32)
    dy = _rand(g, n, D)
    _check_grad(nv.embed_grad(ids.cuda(), dy.cuda(), V), ids, dy, V, 1.0)


@pytest.mark.parametrize("V", [2, 65537, 262143, 262144, 300000])
@pytest.mark.parametrize("n", [100, 17000])
def test_gradient_key_widths(V, n):
    """Vocabularies on both sides of a digit's and a pass's width."""
    say("embed_grad keys", V, n)
    g = torch.Generator().manual_seed(V)
    ids = _ids(g, n, V, "uniform", torch.int64)
    ids[0], ids[-1], ids[1] = V - 1, 0, V
    dy = _rand(g, n, 3)
    _check_grad(nv.embed_grad(ids.cuda(), dy.cuda(), V), ids, dy, V, 1.0)


@pytest.mark.parametrize("D", [1, 511, 520, 1032, 4100])
def test_gradient_widths_and_strides(D):
    say("embed_grad width", D)
    g = torch.Generator().manual_seed(D)
    n, V = 300, 23
    ids = _ids(g, n, V, "zipf", torch.int64)
    for yt, wt in [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16),
                   (torch.bfloat16, torch.float32)]:
        dy = _rand(g, n, D, dtype=yt)
        ws = torch.empty(nv.nvfp4_embed_grad_workspace_bytes(n, V, D), dtype=torch.uint8, device="cuda")
        dw = torch.full((V, D + 3), 5.0, dtype=wt, device="cuda")
        nv.nvfp4_embed_grad(ids.cuda(), _strided(dy, 5, 1), -0.3, dw[:, :D], False, ws)
        _check_grad(dw[:, :D], ids, dy, V, -0.3)
        assert torch.all(dw[:, D:] == 5.0)


@pytest.mark.parametrize("wt", [torch.bfloat16, torch.float32])
def test_gradient_accumulates(wt):
    g = torch.Generator().manual_seed(9)
    n, V, D = 500, 700, 72
    ids, dy = _ids(g, n, V, "zipf", torch.int64), _rand(g, n, D)
    base = _rand(g, V, D, dtype=wt)
    got = base.cuda()
    assert nv.embed_grad(ids.cuda(), dy.cuda(), V, 0.9, accumulate_into=got) is got
    _check_grad(got, ids, dy, V, 0.9, base)
    absent = torch.bincount(ids, minlength=V) == 0
    assert absent.any() and torch.equal(got.cpu()[absent], base[absent])


def test_gradient_is_the_same_every_time():
    g = torch.Generator().manual_seed(4)
    n, V, D = 30001, 1009, 130
    ids, dy = _ids(g, n, V, "zipf", torch.int64).cuda(), _rand(g, n, D).cuda()
    first = nv.embed_grad(ids, dy, V)
    for _ in range(3):
        assert torch.equal(nv.embed_grad(ids, dy, V), first)


def test_gradient_nonfinite_rows_stay_with_their_words():
    ids = torch.tensor([0, 1, 1, 2, -1], device="cuda")
    dy = torch.ones(5, 8, device="cuda")
    dy[1], dy[3], dy[4] = float("inf"), float("nan"), float("nan")
    got = nv.embed_grad(ids, dy, 5).cpu()
    assert torch.all(got[0] == 1) and torch.isinf(got[1]).all() and torch.isnan(got[2]).all()
    assert torch.all(got[3:] == 0)


def test_gradient_on_another_stream_and_in_a_graph():
    g = torch.Generator().manual_seed(5)
    n, V, D = 900, 300, 96
    ids, dy = _ids(g, n, V, "zipf", torch.int64).cuda(), _rand(g, n, D).cuda()
    dw = torch.empty(V, D, device="cuda")
    out = torch.empty(n, D, device="cuda")
    ws = torch.empty(nv.nvfp4_embed_grad_workspace_bytes(n, V, D), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    nv.nvfp4_embed_grad(ids, dy, 1.0, dw, False, ws, stream=side)
    side.synchronize()
    _check_grad(dw, ids.cpu(), dy.cpu(), V, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_embed_grad(ids, dy, 1.0, dw, False, ws)
        nv.nvfp4_embed(ids, dw, 2.0, out)
    for seed in range(3):
        g2 = torch.Generator().manual_seed(100 + seed)
        ids.copy_(_ids(g2, n, V, "zipf", torch.int64))
        dy.copy_(_rand(g2, n, D))
        dw.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        _check_grad(dw, ids.cpu(), dy.cpu(), V, 1.0)
        assert torch.equal(out, nv.embed(ids, dw, 2.0))


@pytest.mark.parametrize("runs", [[16], [17], [15, 1], [1, 15, 16], [16, 48], [16, 49], [64, 64, 1],
                                  [10, 44, 10, 3], [3, 200, 5, 64, 1], [8, 16, 16, 24, 128, 64]])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("D", [5, 8, 515, 1030])
def test_gradient_run_ends(runs, add, D):
    """Runs of one word that end at, before and after the ends of a wave's 16
    rows and of a window of 64, the words absent from the vocabulary among them."""
    say("embed_grad runs", runs, add, D)
    g = torch.Generator().manual_seed(sum(runs) + D)
    V = len(runs) + 2
    for outside in (False, True):
        ids = torch.cat([torch.full((r,), i + 1) for i, r in enumerate(runs)])
        if outside:   # the last run's tokens carry no word
            ids[ids == len(runs)] = V
        order = torch.randperm(len(ids), generator=g)
        ids = ids[order]
        for yt, wt in [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)]:
            dy, base = _rand(g, len(ids), D, dtype=yt), _rand(g, V, D, dtype=wt)
            got = base.cuda() if add else None
            got = nv.embed_grad(ids.cuda(), dy.cuda(), V, 0.7, dtype=wt, accumulate_into=got)
            _check_grad(got, ids, dy, V, 0.7, base if add else None)


@pytest.mark.parametrize("n", [2047, 2048, 2049, 4096, 8191, 8192])
@pytest.mark.parametrize("V,D", [(53, 24), (60001, 420)])
def test_gradient_with_short_and_long_zeros(n, V, D):
    """The two sorts of as many tokens: beside a short and beside a long fill."""
    say("embed_grad fill", n, V, D)
    g = torch.Generator().manual_seed(n + V)
    ids, dy = _ids(g, n, V, "outside", torch.int64), _rand(g, n, D)
    _check_grad(nv.embed_grad(ids.cuda(), dy.cuda(), V), ids, dy, V, 1.0)


def test_lookup_of_more_tokens_than_a_launch_has_threads():
    """2^26 tokens and some: one wave each is 2^32 threads, more than one dimension of
    a launch holds."""
    n, V, D = (1 << 26) + 77, 1000, 8
    say("embed 2^26", n)
    g = torch.Generator().manual_seed(1)
    w = _rand(g, V + 1, D, dtype=torch.bfloat16).cuda()
    w[V] = 0   # what an id outside gives
    ids = torch.arange(n, dtype=torch.int32, device="cuda") % (V + 1)
    out = nv.embed(ids, w[:V])
    for at in range(0, n, 1 << 24):
        assert torch.equal(out[at:at + (1 << 24)], w[ids[at:at + (1 << 24)].long()])


def test_gradient_of_more_tokens_than_a_launch_has_threads():
    """2^30 tokens and some.  Every gradient is 1, so a piece of a sum is a whole number;
    sums of whole windows are multiples of 64 below 2^30, exact in binary32, and only the
    few other pieces round."""
    n, V = (1 << 30) + 130, 3
    say("embed_grad 2^30", n)
    ids = torch.arange(n, dtype=torch.int32, device="cuda") % 4   # a quarter carries no word
    dy = torch.ones(n, 1, dtype=torch.bfloat16, device="cuda")
    got = nv.embed_grad(ids, dy, V, dtype=torch.float32).cpu().double()
    want = torch.tensor([(n - v + 3) // 4 for v in range(V)], dtype=torch.float64).unsqueeze(1)
    assert torch.all((got - want).abs() <= want * 8 * U32), (got, want)


# More than 32768 tokens: the sort in passes over tiles of 4096, with 1 (V <= 511), 2
# and 3 (V >= 2^18) passes, and with histograms of more than the 4096 words that the scan
# takes at a time.
@pytest.mark.parametrize("n", [32769, 40000, 70000])
@pytest.mark.parametrize("V", [300, 511, 131072, 300000])
@pytest.mark.parametrize("kind", ["zipf", "outside"])
def test_gradient_of_many_tokens_and_words(n, V, kind):
    say("embed_grad many words", n, V, kind)
    g = torch.Generator().manual_seed(n + V)
    ids = _ids(g, n, V, kind, torch.int64 if n % 2 else torch.int32)
    ids[0], ids[n // 2], ids[-1] = V - 1, 0, V
    dy = _rand(g, n, 9)
    first = nv.embed_grad(ids.cuda(), dy.cuda(), V, 0.7)
    _check_grad(first, ids, dy, V, 0.7)
    assert torch.equal(nv.embed_grad(ids.cuda(), dy.cuda(), V, 0.7), first)


@pytest.mark.parametrize("V", [300, 131072, 300000])
def test_gradient_of_many_tokens_accumulates(V):
    """More than 32768 tokens added to what dW holds; absent words' rows are not touched."""
    say("embed_grad many, added", V)
    g = torch.Generator().manual_seed(V + 1)
    n = 40001
    ids, dy = _ids(g, n, V, "zipf", torch.int64), _rand(g, n, 9)
    base = _rand(g, V, 9)
    got = nv.embed_grad(ids.cuda(), dy.cuda(), V, 0.9, accumulate_into=base.cuda())
    _check_grad(got, ids, dy, V, 0.9, base)
    absent = torch.bincount(ids, minlength=V) == 0
    assert torch.equal(got.cpu()[absent], base[absent])
