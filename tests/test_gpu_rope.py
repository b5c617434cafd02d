"""The norm and rotation of queries and keys, and the gradient, against float64.

Tolerances, per entry: the row's mean square is an FP32 sum of D squares, relative (D + 2) U at
most (U = 2^-24 per rounding), half of it in its root; z = x r w takes three more, cos and sin
4 steps each (their angle, formed in FP64, is rounded once), the rotation's products and sum two,
of |a| + |b|; one rounding to the result's type (half a step).  The gradient's sums over a row
add D + 4 more of the sum of magnitudes; dw adds up n terms."""
import math

import pytest
import torch

import bit_microscaled_numerics_amd as nv
from parity import say

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24


def _parts(x, rot, il):
    if il:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _join(a, b, rest, il):
    ab = torch.stack((a, b), -1).flatten(-2) if il else torch.cat((a, b), -1)
    return torch.cat((ab, rest), -1)


def _turn(x, cos, sin, rot, il):
    """(rotated, sum of magnitudes)."""
    a, b, rest = _parts(x, rot, il)
    mag = a.abs() * cos.abs() + b.abs() * sin.abs(), b.abs() * cos.abs() + a.abs() * sin.abs()
    size = a.abs() + b.abs()
    return (_join(a * cos - b * sin, b * cos + a * sin, rest, il),
            _join(mag[0] + size, mag[1] + size, rest.abs(), il))


def _angles(pos, inv):
    t = pos.double().unsqueeze(1) * inv.double()
    return torch.cos(t).unsqueeze(1), torch.sin(t).unsqueeze(1)


def _forward(x, w, cos, sin, rot, il, eps, norm):
    D = x.shape[-1]
    z = x.double()
    if norm:
        z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps)
        z = z if w is None else z * w.double()
    y, mag = _turn(z, cos, sin, rot, il)
    return y, (D / 2 + 12) * U * mag


def _gradient(dy, x, w, cos, sin, rot, il, eps, norm):
    D = x.shape[-1]
    dz, mag = _turn(dy.double(), cos, -sin, rot, il)
    e = 8 * U * mag
    if not norm:
        return dz, e, None, None
    n = x.double()
    r = 1 / torch.sqrt((n * n).mean(-1, keepdim=True) + eps)
    n = n * r
    rel = (D / 2 + 4) * U
    wd = torch.ones(D, dtype=torch.float64) if w is None else w.double()
    dn = dz * wd
    m = (dn * n).mean(-1, keepdim=True)
    dx = r * (dn - n * m)
    m_err = ((e * wd.abs() * n.abs()).mean(-1, keepdim=True)
             + ((D + 4) * U + 2 * rel) * (dn * n).abs().mean(-1, keepdim=True))
    dx_err = r * (e * wd.abs() + 2 * U * dn.abs() + n.abs() * (m_err + (2 * rel + 3 * U) * m.abs())) \
        + rel * (r * (dn.abs() + (n * m).abs()))
    rows = dz.numel() // D
    dw = (dz * n).sum((0, 1))
    dw_err = (e * n.abs()).sum((0, 1)) + (rel + (rows + 8) * U) * (dz * n).abs().sum((0, 1))
    return dx, dx_err, dw, dw_err


def _close(got, want, err, dtype, name):
    tol = err * (1 + HALF[dtype]) + HALF[dtype] * want.abs() + 1e-40
    bad = (got.cpu().double() - want).abs() > tol
    assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:3].tolist(),
                           got.cpu().double()[bad][:3].tolist(), want[bad][:3].tolist())


def _inv(rot, base=1e4):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float()


CASES = [  # T, Hq, Hkv, D, rot
    (1, 32, 8, 128, 128), (1, 1, 1, 2, 2), (0, 4, 2, 64, 64), (5, 0, 3, 16, 16), (33, 3, 0, 64, 32),
    (257, 6, 2, 80, 36), (19, 5, 5, 512, 512), (77, 12, 4, 64, 64), (3, 40, 8, 128, 64), (130, 2, 1, 34, 0),
    (1000, 2, 1, 96, 96), (4, 65, 3, 256, 160), (50, 7, 7, 22, 10)]


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("dt,wt", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                   (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", CASES)
def test_against_float64(T, Hq, Hkv, D, rot, dt, wt, il):
    say("rope", T, Hq, Hkv, D, rot, dt, wt, il)
    g = torch.Generator().manual_seed(T + D)
    eps, norm = 1e-6, (T + D) % 5 != 0
    q, k, dq, dk = (torch.randn(T, H, D, generator=g).to(dt) for H in (Hq, Hkv, Hq, Hkv))
    wq = (1 + 0.3 * torch.randn(D, generator=g)).to(wt) if norm else None
    wk = (1 + 0.3 * torch.randn(D, generator=g)).to(wt) if norm and D != 34 else None
    pos = torch.randint(-50, 200000, (T,), generator=g).to(torch.int64 if D % 4 else torch.int32)
    inv = _inv(rot)
    c = lambda x: None if x is None else x.cuda()
    args = (c(q), c(k), c(wq), c(wk)) + ((c(pos), c(inv)) if rot else (None, None))
    kw = dict(eps=eps, interleaved=il, norm=norm)
    qo, ko = nv.qk_norm_rope(*args, **kw)
    dqi, dki, dwq, dwk = nv.qk_norm_rope_grad(c(dq), c(dk), *args, **kw)
    cos, sin = _angles(pos, inv)
    for x, w, dy, y, dx, dw, name in ((q, wq, dq, qo, dqi, dwq, "q"), (k, wk, dk, ko, dki, dwk, "k")):
        want, err = _forward(x, w, cos, sin, rot, il, eps, norm)
        _close(y, want, err, dt, name)
        dx_w, dx_e, dw_w, dw_e = _gradient(dy, x, w, cos, sin, rot, il, eps, norm)
        _close(dx, dx_w, dx_e, dt, "d" + name)
        assert (dw is None) == (w is None)
        if w is not None:
            assert dw.dtype == w.dtype and dw.shape == w.shape
            _close(dw, dw_w, dw_e, wt, "dw" + name)


def test_far_positions():
    """Angles of far positions are those of the definition, to the FP32 of their cosine."""
    say("rope far")
    pos = torch.tensor([0, 1, 2 ** 20 + 1, 2 ** 24 + 3, 2 ** 29 - 1, -(2 ** 29) + 7])
    inv = _inv(64, 5e5)
    q = torch.zeros(6, 1, 64)
    q[..., :32] = 1.0
    y, _ = nv.qk_norm_rope(q.cuda(), q[:, :0].cuda(), positions=pos.cuda(), inv_freq=inv.cuda(), norm=False)
    t = pos.double().unsqueeze(1) * inv.double()   # below 2^53: exact
    # the float64 cosine's own argument is exact; two roundings and the functions' 4 steps
    assert ((y[:, 0, :32].cpu().double() - torch.cos(t)).abs() <= 8 * U).all()
    assert ((y[:, 0, 32:].cpu().double() - torch.sin(t)).abs() <= 8 * U).all()


@pytest.mark.parametrize("dt,lead", [(torch.bfloat16, 0), (torch.bfloat16, 1), (torch.float32, 3)])
def test_strides_and_in_place(dt, lead):
    """Pieces of a projection's rows, at any element; in place; nothing beside them."""
    say("rope strides", dt, lead)
    g = torch.Generator().manual_seed(1)
    T, Hq, Hkv, D = 70, 5, 2, 48
    q, k, dq, dk = (torch.randn(T, H, D, generator=g).to(dt).cuda() for H in (Hq, Hkv, Hq, Hkv))
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    pos, inv = torch.arange(T, device="cuda", dtype=torch.int32), _inv(32).cuda()
    want = nv.qk_norm_rope(q, k, w, w, pos, inv)
    want_g = nv.qk_norm_rope_grad(dq, dk, q, k, w, w, pos, inv)
    width = (Hq + 2 * Hkv) * D + 5

    def fused(a, b):
        buf = torch.full((T, width), 3.0, dtype=dt, device="cuda")
        x = buf[:, lead:lead + Hq * D].view(T, Hq, D)
        y = buf[:, lead + Hq * D:lead + (Hq + Hkv) * D].view(T, Hkv, D)
        x.copy_(a)
        y.copy_(b)
        return buf, x, y

    buf, x, y = fused(q, k)
    assert all(torch.equal(a, b) for a, b in zip(nv.qk_norm_rope(x, y, w, w, pos, inv), want))
    gbuf, dx, dy = fused(dq, dk)
    got = nv.qk_norm_rope_grad(dx, dy, x, y, w, w, pos, inv, out=(dx, dy))
    assert all(torch.equal(a, b) for a, b in zip(got, want_g))
    nv.nvfp4_qk_norm_rope(x, y, w, w, pos, inv, 1e-6, False, True, x, y)
    assert torch.equal(x, want[0]) and torch.equal(y, want[1])
    for b in (buf, gbuf):
        assert torch.all(b[:, lead + (Hq + Hkv) * D:] == 3.0) and torch.all(b[:, :lead] == 3.0)
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(nv.qk_norm_rope(heads_first, k, w, w, pos, inv)[0], want[0])


def test_rows_that_are_not_finite_stay_alone():
    say("rope not finite")
    g = torch.Generator().manual_seed(2)
    q, k = torch.randn(20, 3, 64, generator=g).cuda(), torch.randn(20, 2, 64, generator=g).cuda()
    pos, inv = torch.arange(20, device="cuda"), _inv(64).cuda()
    want = nv.qk_norm_rope(q, k, positions=pos, inv_freq=inv)
    q[3, 1, 5], k[7, 0, 0] = float("nan"), float("inf")
    got = nv.qk_norm_rope(q, k, positions=pos, inv_freq=inv)
    for a, b, bad in zip(got, want, ((3, 1), (7, 0))):
        keep = torch.ones(a.shape[:2], dtype=torch.bool, device="cuda")
        keep[bad] = False
        assert torch.equal(a[keep], b[keep])


def test_many_tokens_and_same_bits():
    say("rope many tokens")
    g = torch.Generator().manual_seed(3)
    T, Hq, Hkv, D = 20000, 4, 1, 64
    q, k, dq, dk = (torch.randn(T, H, D, generator=g).to(torch.bfloat16) for H in (Hq, Hkv, Hq, Hkv))
    w = (1 + 0.1 * torch.randn(D, generator=g))
    pos, inv = torch.arange(T) % 4096, _inv(D)
    args = tuple(x.cuda() for x in (dq, dk, q, k, w, w, pos, inv))
    got = nv.qk_norm_rope_grad(*args)
    cos, sin = _angles(pos, inv)
    for i, (x, dy) in enumerate(((q, dq), (k, dk))):
        dx, dx_e, dw, dw_e = _gradient(dy, x, w, cos, sin, D, False, 1e-6, True)
        _close(got[i], dx, dx_e, torch.bfloat16, "dx")
        _close(got[2 + i], dw, dw_e, torch.float32, "dw")
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(nv.qk_norm_rope_grad(*args), got))


def test_gradient_against_differences():
    say("rope differences")
    g = torch.Generator().manual_seed(4)
    T, H, D, rot = 9, 2, 24, 16
    q, dq = torch.randn(T, H, D, generator=g), torch.randn(T, H, D, generator=g)
    w, pos, inv = 1 + 0.2 * torch.randn(D, generator=g), torch.arange(T) * 37, _inv(rot)
    e = q[:, :0]
    dx, _, dw, _ = nv.qk_norm_rope_grad(*(x.cuda() for x in (dq, e, q, e, w, w, pos, inv)), interleaved=True)
    cos, sin = _angles(pos, inv)

    def loss(x, ww):
        return float((_forward(x, ww, cos, sin, rot, True, 1e-6, True)[0] * dq.double()).sum())

    for got, at in ((dx, 0), (dw, 1)):
        args = [q.double(), w.double()]
        way = torch.randn(*got.shape, generator=g, dtype=torch.float64)
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + 1e-6 * way, args[at] - 1e-6 * way
        diff = (loss(*up) - loss(*down)) / 2e-6
        mine = float((got.cpu().double() * way).sum())
        # FP32 sums of T H D terms of size about 1, and the differences' own error
        assert abs(mine - diff) <= 2 ** -20 * math.sqrt(T * H * D) * 8 + 1e-7 * abs(diff)


def test_replayed_graph():
    say("rope graph")
    g = torch.Generator().manual_seed(5)
    q, k, dq, dk = (torch.randn(333, H, 64, generator=g).to(torch.bfloat16).cuda() for H in (4, 2, 4, 2))
    w, inv = torch.ones(64, device="cuda"), _inv(64).cuda()
    pos = torch.arange(333, device="cuda")

    def step():
        return (*nv.qk_norm_rope(q, k, w, w, pos, inv), *nv.qk_norm_rope_grad(dq, dk, q, k, w, w, pos, inv))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        for x in (q, k, dq, dk):
            x.normal_()
        pos.add_(1000)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))
