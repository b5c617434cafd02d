"""Values that are not finite, against the definition taken pair by pair: what a query sees makes its results
NaN or infinite as the formulas do, what it does not see changes nothing, and a step of such values takes no
longer than a small multiple of an ordinary one."""
import pytest
import torch

import attn_reference as ref
import bit_microscaled_numerics_amd as nv
from parity import say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
NAN, INF = float("nan"), float("inf")


def _rand(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(BF).cuda()


def _by_pairs(q, k, v, dout, seen, scale):
    """Float64 (out, lse, dq, dk, dv) of [tokens][heads][D] operands, every sum over seen pairs alone."""
    q, k, v, dout = (x.double().cpu() for x in (q, k, v, dout))
    G = q.shape[1] // k.shape[1]
    out, dq, dk, dv = (torch.zeros_like(x) for x in (q, q, k, v))
    lse = torch.full(q.shape[:2], -INF, dtype=torch.float64)
    some, pairs = seen.any(1), seen.unsqueeze(2)
    zero = torch.zeros((), dtype=torch.float64)
    for h in range(q.shape[1]):
        qh, kh, vh, gh = q[:, h], k[:, h // G], v[:, h // G], dout[:, h]
        # products that are not seen are looked at nowhere: a sum takes zeros in their place
        s = scale * (qh.unsqueeze(1) * kh.unsqueeze(0)).sum(2)
        top = torch.where(seen, s, -INF).max(1, keepdim=True).values
        top = torch.where((seen & torch.isnan(s)).any(1, keepdim=True), NAN, top)
        e = torch.where(seen, torch.exp(s - top), zero)   # NaN throughout from an infinite score on
        total = e.sum(1, keepdim=True)
        p = torch.where(seen, e / total, zero)
        lse[some, h] = (top + torch.log(total))[some, 0]
        out[:, h] = torch.where(pairs, p.unsqueeze(2) * vh, zero).sum(1)
        delta = (gh * out[:, h]).sum(1, keepdim=True)
        ds = torch.where(seen, p * ((gh.unsqueeze(1) * vh).sum(2) - delta), zero)
        dv[:, h // G] += torch.where(pairs, p.unsqueeze(2) * gh.unsqueeze(1), zero).sum(0)
        dq[:, h] = scale * torch.where(pairs, ds.unsqueeze(2) * kh, zero).sum(1)
        dk[:, h // G] += scale * torch.where(pairs, ds.unsqueeze(2) * qh.unsqueeze(1), zero).sum(0)
    return out, lse, dq, dk, dv


def _check(q, k, v, dout, clean, seen, T, **kw):
    """Finite where the definition is, and there within the bound of the clean operands if nothing
    that differs from them reaches the row; not finite where it is not."""
    out, lse = nv.attention(q, k, v, **kw)
    got = (out, lse, *nv.attention_grad(dout, q, k, v, out, lse, **kw))
    want = _by_pairs(q, k, v, dout, seen, q.shape[-1] ** -0.5)
    plain = _by_pairs(*clean, seen, q.shape[-1] ** -0.5)
    for name, a, b, c in zip(("out", "lse", "dq", "dk", "dv"), got, want, plain):
        a = a.double().cpu()
        finite = torch.isfinite(b) | (b == -INF) if name == "lse" else torch.isfinite(b)
        assert torch.isnan(a)[torch.isnan(b)].all(), (name, "NaN lost")
        assert not torch.isnan(a)[finite].any(), (name, int(torch.isnan(a)[finite].sum()))
        if name != "lse":
            assert torch.isfinite(a)[finite].all(), name
            assert not torch.isfinite(a)[torch.isinf(b)].any(), (name, "infinity lost")
        same = (b == c) | (finite & ((b - c).abs() <= 1e-12))
        # p and ds rounded to BF16, the result once, delta from the rounded out: four half steps of the size
        # of the largest entries of the tensor are far above what a wrong row would be below
        size = 4 * 2.0 ** -8 * max(1.0, float(torch.nan_to_num(c, posinf=0, neginf=0).abs().max()))
        assert ((a - c).abs()[same & torch.isfinite(c)] <= size).all(), (name, float((a - c).abs()[same & torch.isfinite(c)].max()))


PLACES = ["one", "row", "rows", "all"]


@pytest.mark.parametrize("which", [0, 1, 2, 3])
@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("mask", ["causal", "window", "packed", "both"])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(150, 2, 1, 64), (70, 3, 3, 128), (200, 4, 1, 24)])
def test_by_pairs(T, Hq, Hkv, D, mask, value, place, which):
    say("attention not finite", T, Hq, Hkv, D, mask, value, place, which)
    g = torch.Generator().manual_seed(T + which)
    q, k, v, dout = (_rand(g, T, H, D) for H in (Hq, Hkv, Hkv, Hq))
    clean = [x.clone() for x in (q, k, v, dout)]
    x = (q, k, v, dout)[which]
    if place == "one":
        x[T // 2, 0, D // 3] = value
    elif place == "row":
        x[T // 2, 0] = value
    elif place == "rows":
        x[T // 3::7, -1] = value
    else:
        x.fill_(value)
    kw = dict(causal=mask != "both", window=40 if mask == "window" else 0)
    seen = ref.seen_mask(T, T, kw["causal"], kw["window"])
    if mask == "packed":
        cu = [0, T // 4, T // 4 + 1, T // 2 + 3, T - 5]   # tokens behind the last
        kw["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        seen = torch.zeros(T, T, dtype=torch.bool)
        for a, b in zip(cu, cu[1:]):
            seen[a:b, a:b] = ref.seen_mask(b - a, b - a, True, 0)
    _check(q, k, v, dout, clean, seen, T, **kw)


@pytest.mark.parametrize("Tk", [700, 5000])
@pytest.mark.parametrize("which", [1, 2])
def test_few_queries(Tk, which):
    """The joins of parts: a part whose scores are all NaN, and one NaN among many parts."""
    say("attention not finite, parts", Tk, which)
    g = torch.Generator().manual_seed(Tk)
    Tq, Hq, D = 2, 4, 64
    for bad in (slice(0, Tk), slice(130, 460), slice(Tk - 1, Tk)):
        q, k, v, dout = (_rand(g, T, H, D) for T, H in ((Tq, Hq), (Tk, 1), (Tk, 1), (Tq, Hq)))
        clean = [x.clone() for x in (q, k, v, dout)]
        (k, v)[which - 1][bad] = NAN
        _check(q, k, v, dout, clean, ref.seen_mask(Tq, Tk, True, 0), Tq, causal=True)


def _us(f):
    f()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(True), torch.cuda.Event(True)
    a.record()
    f()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) * 1e3


@pytest.mark.parametrize("which", ["qkv", "q", "k", "v", "dout", "token"])
def test_a_diverged_step_ends_soon(which):
    """Ordinary work of 4096 tokens takes some 100 us; formed pair by pair it would be hundreds of times that.
    Twenty times leaves room for the card's clocks."""
    say("attention diverged", which)
    g = torch.Generator().manual_seed(3)
    ops = dict(q=_rand(g, 4096, 8, 128), k=_rand(g, 4096, 2, 128), v=_rand(g, 4096, 2, 128),
               dout=_rand(g, 4096, 8, 128))

    def times(q, k, v, dout):
        out, lse = nv.attention(q, k, v, causal=True)
        return (_us(lambda: nv.attention(q, k, v, causal=True)),
                _us(lambda: nv.attention_grad(dout, q, k, v, out, lse, causal=True)))

    usual = times(**ops)
    for name, x in ops.items():
        if name in which:
            x.fill_(NAN)
        elif which == "token" and name in "qkv":
            x[100] = NAN
    for got, was in zip(times(**ops), usual):
        assert got <= 20 * max(was, 50.0), (got, was)
