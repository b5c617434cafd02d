"""Attention and its gradient against float64, entry by entry within the bounds that
tests/attn_reference.py derives: lengths from one token on, odd sizes, head groups,
strides, masks that leave rows empty, packed sequences, values that a mask hides."""
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
    got = got.double()
    same = got == want   # infinities and exact zeros
    bad = ~(same | ((got - want).abs() <= tol))
    assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           got[bad][:4].tolist(), want[bad][:4].tolist(), tol[bad][:4].tolist())


def _check(q, k, v, dout, causal=False, window=0, cu=None, scale=None):
    """Forward and gradient of one call against float64."""
    kw = dict(scale=scale, causal=causal, window=window)
    bounds = None
    if cu is not None:
        cu_q, cu_k, it = cu
        bounds = list(zip(cu_q, cu_q[1:], cu_k, cu_k[1:]))
        kw.update(cu_q=torch.tensor(cu_q, dtype=it, device="cuda"),
                  cu_k=torch.tensor(cu_k, dtype=it, device="cuda"))
    out, lse = nv.attention(q, k, v, **kw)
    grads = nv.attention_grad(dout, q, k, v, out, lse, **kw)
    sc = q.shape[-1] ** -0.5 if scale is None else scale
    r, t = ref.attention(q, k, v, sc, causal, window, bounds, dout)
    for name, x in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        assert x.shape == r[name].shape
        _close(x, r[name], t[name], name)
    return out, lse, grads


SHAPES = [  # B, Tq, Tk, Hq, Hkv, D
    (1, 1, 1, 1, 1, 8), (1, 1, 300, 8, 2, 64), (2, 3, 5, 4, 4, 16), (1, 64, 64, 2, 1, 32),
    (1, 65, 63, 3, 1, 40), (2, 127, 129, 4, 2, 128), (1, 128, 128, 6, 2, 96), (1, 257, 257, 5, 5, 72),
    (1, 31, 700, 2, 2, 128), (1, 500, 33, 2, 1, 64), (3, 130, 130, 7, 1, 80), (1, 900, 900, 2, 1, 128),
    (1, 0, 5, 2, 1, 32), (1, 5, 0, 2, 1, 32), (0, 4, 4, 2, 1, 32)]


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 1), (True, 50), (True, 200)])
@pytest.mark.parametrize("B,Tq,Tk,Hq,Hkv,D", SHAPES)
def test_against_float64(B, Tq, Tk, Hq, Hkv, D, causal, window):
    say("attention", B, Tq, Tk, Hq, Hkv, D, causal, window)
    g = torch.Generator().manual_seed(Tq * 1000 + Tk + D)
    _check(_rand(g, B, Tq, Hq, D, std=1.3), _rand(g, B, Tk, Hkv, D, std=1.3), _rand(g, B, Tk, Hkv, D),
           _rand(g, B, Tq, Hq, D), causal, window)


@pytest.mark.parametrize("T,H,D", [(2500, 2, 128), (3001, 1, 64)])
def test_long(T, H, D):
    say("attention long", T, H, D)
    g = torch.Generator().manual_seed(T)
    _check(_rand(g, T, 2 * H, D), _rand(g, T, H, D), _rand(g, T, H, D), _rand(g, T, 2 * H, D), True)


@pytest.mark.parametrize("Tq,Tk,Hq,Hkv,D", [(1, 20000, 8, 1, 128), (1, 9001, 4, 4, 64), (7, 5000, 6, 2, 80),
                                            (40, 6000, 2, 1, 128)])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 3001)])
def test_few_queries_over_many_keys(Tq, Tk, Hq, Hkv, D, causal, window):
    say("attention few", Tq, Tk, Hq, Hkv, D, causal, window)
    g = torch.Generator().manual_seed(Tq + Tk)
    _check(_rand(g, 2, Tq, Hq, D), _rand(g, 2, Tk, Hkv, D), _rand(g, 2, Tk, Hkv, D), _rand(g, 2, Tq, Hq, D),
           causal, window)


LENGTHS = [
    ([7, 1, 0, 64, 130, 0, 3, 257], None, 9),              # tokens behind the last sequence
    ([1] * 300, None, 0),
    ([0, 0, 5, 0], None, 0),
    ([200, 0, 31, 65], [180, 12, 0, 400], 3),              # other keys than queries; one has none
    ([5, 90, 1], [700, 1, 1000], 0),
    ([], None, 4)]


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 40)])
@pytest.mark.parametrize("it", [torch.int32, torch.int64])
@pytest.mark.parametrize("nq,nk,extra", LENGTHS)
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (3, 1, 128)])
def test_packed(nq, nk, extra, it, causal, window, Hq, Hkv, D):
    nk = nq if nk is None else nk
    say("attention packed", nq[:4], nk[:4], extra, it, causal, window, Hq, Hkv, D)
    cu = [[sum(n[:i]) for i in range(len(n) + 1)] for n in (nq, nk)]
    g = torch.Generator().manual_seed(sum(nq))
    Tq, Tk = sum(nq) + extra, sum(nk) + extra
    # what lies behind the last sequence reaches nothing
    q, k, v, dout = (_rand(g, T, H, D) for T, H in ((Tq, Hq), (Tk, Hkv), (Tk, Hkv), (Tq, Hq)))
    for x, n in ((q, nq), (k, nk), (v, nk), (dout, nq)):
        x[sum(n):] = float("nan")
    kw = dict(causal=causal, window=window, cu_q=torch.tensor(cu[0], dtype=it, device="cuda"),
              cu_k=torch.tensor(cu[1], dtype=it, device="cuda"))
    out, lse = nv.attention(q, k, v, **kw)
    grads = nv.attention_grad(dout, q, k, v, out, lse, **kw)
    qz, kz, vz, dz = (torch.nan_to_num(x) for x in (q, k, v, dout))
    r, t = ref.attention(qz, kz, vz, D ** -0.5, causal, window,
                         list(zip(cu[0], cu[0][1:], cu[1], cu[1][1:])), dz)
    for name, x in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        _close(x, r[name], t[name], name)


@pytest.mark.parametrize("n", [1, 62, 63, 64, 65, 127, 128, 129, 500])
def test_number_of_sequences(n):
    """The sequence of a row is found whatever their number, with empty ones at both ends and between."""
    say("attention sequences", n)
    g = torch.Generator().manual_seed(n)
    lengths = torch.randint(0, 6, (2, n), generator=g)
    lengths[:, :min(2, n - 1)] = 0
    lengths[:, n - 1] *= n % 2
    cu = torch.cat((torch.zeros(2, 1, dtype=torch.int64), lengths.cumsum(1)), 1).tolist()
    (Tq, Tk), Hq, Hkv, D = (c[-1] + 2 for c in cu), 2, 1, 64
    _check(_rand(g, Tq, Hq, D), _rand(g, Tk, Hkv, D), _rand(g, Tk, Hkv, D), _rand(g, Tq, Hq, D), n % 4 == 1,
           cu=(*cu, torch.int32 if n % 2 else torch.int64))


def _view(x, kind):
    """The same values in another layout."""
    B, T, H, D = x.shape
    if kind == "heads_first":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if kind == "tokens_first":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    buf = torch.full((B, T, 3 * H * D + 24), 9.0, dtype=BF, device="cuda")   # a projection's rows
    v = buf[..., 8:8 + H * D].view(B, T, H, D)
    v.copy_(x)
    return v


@pytest.mark.parametrize("kind", ["heads_first", "tokens_first", "fused"])
def test_layouts(kind):
    say("attention layouts", kind)
    g = torch.Generator().manual_seed(5)
    B, T, Hq, Hkv, D = 2, 150, 4, 2, 72
    q, k, v, dout = (_rand(g, B, T, H, D) for H in (Hq, Hkv, Hkv, Hq))
    out, lse = nv.attention(q, k, v, causal=True)
    grads = nv.attention_grad(dout, q, k, v, out, lse, causal=True)
    q2, k2, v2, d2, o2 = (_view(x, kind) for x in (q, k, v, dout, torch.zeros_like(q)))
    l2 = torch.empty_like(lse)
    a = nv._attn(q2, k2, v2, None, True, 0, None, None)[0]
    ws = torch.empty(max(1, nv.nvfp4_attention_workspace_bytes(a, False)), dtype=torch.uint8, device="cuda")
    nv.nvfp4_attention(q2, k2, v2, None, True, 0, None, None, o2, l2, ws)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    g2 = tuple(_view(torch.zeros_like(x), kind) for x in (q, k, v))
    got = nv.attention_grad(d2, q2, k2, v2, o2, l2, causal=True, grads=g2)
    for x, y, z in zip(got, grads, g2):
        assert torch.equal(x, y) and x.data_ptr() == z.data_ptr()
        if kind == "fused":   # nothing beside the rows is written
            assert torch.all(z._base[..., :8] == 9.0) and torch.all(z._base[..., 8 + z.shape[2] * D:] == 9.0)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 30)])
def test_hidden_values_reach_nothing(value, causal, window):
    """Values at one token reach the queries that see it (their out is that of the
    definition) and no other row."""
    say("attention hidden", value, window)
    g = torch.Generator().manual_seed(2)
    T, D, bad = 200, 64, 77
    for which in range(4):
        q, k, v, dout = (_rand(g, T, H, D) for H in (2, 1, 1, 2))
        clean = [x.clone() for x in (q, k, v, dout)]
        (q, k, v, dout)[which][bad] = value
        out, lse = nv.attention(q, k, v, causal=causal, window=window)
        grads = nv.attention_grad(dout, q, k, v, out, lse, causal=causal, window=window)
        r, t = ref.attention(*clean[:3], D ** -0.5, causal, window, None, clean[3])
        seen = ref.seen_mask(T, T, causal, window)
        sees_bad = torch.zeros(T, dtype=torch.bool)   # queries whose row may change
        if which in (1, 2):
            sees_bad = seen[:, bad].clone()
        elif which == 0:
            sees_bad[bad] = True
        free = (~sees_bad).cuda()
        _close(out[free], r["out"][free], t["out"][free], "out")
        _close(lse[free], r["lse"][free], t["lse"][free], "lse")
        if which == 2:
            assert not torch.isfinite(out[~free]).any()
        if which == 3:
            free[bad] = False
        _close(grads[0][free], r["dq"][free], t["dq"][free], "dq")
        touched = seen[~free.cpu()].any(0).cuda()   # keys that a changed query sees
        _close(grads[1][~touched], r["dk"][~touched], t["dk"][~touched], "dk")
        _close(grads[2][~touched], r["dv"][~touched], t["dv"][~touched], "dv")


def test_large_scores_and_scale():
    """Scores up to several hundred: the running maximum keeps the sums finite."""
    say("attention large scores")
    g = torch.Generator().manual_seed(3)
    q, k, v, dout = (_rand(g, 300, 2, 64, std=s) for s in (6.0, 6.0, 1.0, 1.0))
    _check(q, k, v, dout, True, scale=1.0)
    _check(q, k, v, dout, False, scale=1e-3)


@pytest.mark.parametrize("power", [-64, 64])
def test_largest_and_smallest_scale(power):
    say("attention scale", power)
    g = torch.Generator().manual_seed(power + 100)
    std = 1.0 if power < 0 else 2.0 ** -33
    q, k, v, dout = (_rand(g, 150, 2, 64, std=s) for s in (std, std, 1.0, 1.0))
    _check(q, k, v, dout, True, scale=2.0 ** power)


def test_same_bits_every_time():
    say("attention repeat")
    g = torch.Generator().manual_seed(4)
    q, k, v, dout = (_rand(g, 2, 400, H, 128) for H in (6, 2, 2, 6))
    out, lse = nv.attention(q, k, v, causal=True)
    grads = nv.attention_grad(dout, q, k, v, out, lse, causal=True)
    for _ in range(3):
        o2, l2 = nv.attention(q, k, v, causal=True)
        g2 = nv.attention_grad(dout, q, k, v, o2, l2, causal=True)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
        assert all(torch.equal(x, y) for x, y in zip(g2, grads))


def test_gradient_against_differences():
    """dq, dk, dv against central differences of the float64 forward along random directions;
    the kernel's gradient is within its bound of the true one, so their products are too."""
    say("attention differences")
    g = torch.Generator().manual_seed(6)
    T, D = 70, 32
    q, k, v, dout = (_rand(g, T, H, D) for H in (2, 1, 1, 2))
    out, lse = nv.attention(q, k, v, causal=True)
    grads = nv.attention_grad(dout, q, k, v, out, lse, causal=True)
    _, tol = ref.attention(q, k, v, D ** -0.5, True, 0, None, dout)

    def loss(*x):
        r, _ = ref.attention(*x, D ** -0.5, True, 0)
        return float((r["out"] * dout.double()).sum())

    for i, name in enumerate(("dq", "dk", "dv")):
        way = torch.randn(*grads[i].shape, generator=g, dtype=torch.float64).cuda()
        h, args = 1e-5, [q.double(), k.double(), v.double()]
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * way, args[i] - h * way
        diff = (loss(*up) - loss(*down)) / (2 * h)
        got = float((grads[i].double() * way).sum())
        assert abs(got - diff) <= float((tol[name] * way.abs()).sum()) + 1e-6 * abs(diff)


def test_replayed_graph_and_streams():
    """A captured forward and gradient, replayed with other inputs, on a stream of its own."""
    say("attention graph")
    g = torch.Generator().manual_seed(8)
    q, k, v, dout = (_rand(g, 190, H, 64) for H in (4, 2, 2, 4))
    nv.attention_grad(dout, q, k, v, *nv.attention(q, k, v, causal=True), causal=True)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out, lse = nv.attention(q, k, v, causal=True)
        grads = nv.attention_grad(dout, q, k, v, out, lse, causal=True)
    for _ in range(4):
        for x in (q, k, v, dout):
            x.copy_(_rand(g, *x.shape))
        graph.replay()
        torch.cuda.synchronize()
        o2, l2 = nv.attention(q, k, v, causal=True)
        g2 = nv.attention_grad(dout, q, k, v, o2, l2, causal=True)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
        assert all(torch.equal(x, y) for x, y in zip(g2, grads))


@pytest.mark.parametrize("D", [88, 96, 104])
def test_widths_between_the_tiles(D):
    say("attention width", D)
    g = torch.Generator().manual_seed(D)
    _check(_rand(g, 1, 300, 4, D), _rand(g, 1, 300, 2, D), _rand(g, 1, 300, 2, D), _rand(g, 1, 300, 4, D), True)


def test_offsets_past_32_bits():
    """Keys and values 2^22 - 8 elements apart: the last ones lie more than 2^33 bytes in."""
    say("attention far offsets")
    T, D, stride = 1100, 64, (1 << 22) - 8
    g = torch.Generator().manual_seed(11)
    flat = torch.empty(T * stride, dtype=BF, device="cuda")
    far = flat.view(T, stride)
    q, k, v, dout = (_rand(g, T, 1, D) for _ in range(4))
    views = [far[:, i * D:(i + 1) * D].unsqueeze(1) for i in range(3)]
    for x, y in zip(views, (q, k, v)):
        x.copy_(y)
    out, lse = nv.attention(q, k, v, causal=True)
    grads = nv.attention_grad(dout, q, k, v, out, lse, causal=True)
    o2, l2 = nv.attention(*views, causal=True)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    to = tuple(far[:, (3 + i) * D:(4 + i) * D].unsqueeze(1) for i in range(3))
    g2 = nv.attention_grad(dout, *views, out, lse, causal=True, grads=to)
    assert all(torch.equal(x, y) for x, y in zip(g2, grads))


def test_many_heads_of_one_key_head():
    """300 query heads on one key head, more than a step of rows; two calls at once on two streams."""
    say("attention many heads")
    g = torch.Generator().manual_seed(12)
    q, k, v, dout = (_rand(g, 20, H, 32) for H in (300, 1, 1, 300))
    out, lse, grads = _check(q, k, v, dout, True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            o, l = nv.attention(q, k, v, causal=True)
            got.append((o, l, *nv.attention_grad(dout, q, k, v, o, l, causal=True)))
    torch.cuda.synchronize()
    for x in got:
        assert all(torch.equal(a, b) for a, b in zip(x, (out, lse, *grads)))


def test_nothing_finite():
    """A step that has diverged: every value NaN, results NaN, every loop ends."""
    say("attention all NaN")
    x = torch.full((400, 2, 64), float("nan"), dtype=BF, device="cuda")
    out, lse = nv.attention(x, x, x, causal=True)
    grads = nv.attention_grad(x, x, x, x, out, lse, causal=True)
    assert all(torch.isnan(y).all() for y in (out, lse, *grads))


@pytest.mark.parametrize("cu", [[5, 2, 9, 40], [0, 1000, 30, 50], [-7, 20, 10, 50], [3, 50, 50, 50]])
def test_sequence_bounds_that_make_no_sense_stay_inside(cu):
    """Unspecified results, but none outside the operands (the outputs' guard bands) and no
    endless loop."""
    say("attention cu", cu)
    g = torch.Generator().manual_seed(13)
    q, k, v, dout = (_rand(g, 50, H, 64) for H in (2, 1, 1, 2))
    b = torch.tensor(cu, dtype=torch.int64, device="cuda")
    out, lse = nv.attention(q, k, v, causal=True, cu_q=b)
    nv.attention_grad(dout, q, k, v, out, lse, causal=True, cu_q=b)
    torch.cuda.synchronize()


def test_shared_out_parts_of_keys_with_hidden_values():
    """Few queries over many keys and few keys under many queries: the parts' joins, with values
    that only some rows see."""
    say("attention parts")
    g = torch.Generator().manual_seed(14)
    q, k, v, dout = (_rand(g, T, H, 64) for T, H in ((3, 4), (3000, 2), (3000, 2), (3, 4)))
    r, t = ref.attention(q, k, v, 0.125, True, 0, None, dout)
    v[2999] = float("inf")   # only the last query sees it
    out, lse = nv.attention(q, k, v, causal=True)
    _close(out[:2], r["out"][:2], t["out"][:2], "out")
    _close(lse, r["lse"], t["lse"], "lse")
    assert not torch.isfinite(out[2]).any()
    q, k, v, dout = (_rand(g, T, H, 64) for T, H in ((2000, 8), (2000, 1), (2000, 1), (2000, 8)))
    r, t = ref.attention(q, k, v, 0.125, True, 0, None, dout)
    out, lse = nv.attention(q, k, v, causal=True)
    dout[700, 3] = float("nan")   # keys behind token 700 do not see it
    dq, dk, dv = nv.attention_grad(dout, q, k, v, out, lse, causal=True)
    _close(dk[701:], r["dk"][701:], t["dk"][701:], "dk")
    _close(dv[701:], r["dv"][701:], t["dv"][701:], "dv")
    assert torch.isnan(dv[:701]).all()
    keep = torch.ones(2000, 8, dtype=torch.bool, device="cuda")
    keep[700, 3] = False
    _close(dq[keep], r["dq"][keep], t["dq"][keep], "dq")
