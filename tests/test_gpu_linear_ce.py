"""Softmax cross entropy of an output head, and its gradient, against binary64.

Tolerances, from the arithmetic (u = 2^-24, one binary32 rounding):
  logit     products of BF16 are exact in binary32; a sum of D of them is within
            dz = D u sum_k |h_k w_k| of the exact one
  lse       each exponential within dz plus 4 u; a span's sum adds 72 terms in
            sequence and tree, the spans' sum S / 64 + 8 more: relative
            (80 + S / 64 + 8) u, and the result is rounded once
  d         the code is within half a step of 64/65535 in log2: 3.4e-4; dz and
            the lse error enter as relative errors; BF16 rounds by half a step,
            2^-8.  At the target exp(-loss) - 1 takes the loss's error times
            exp(-loss) instead of the code's.
  dh, dw    the errors of d through the product, a binary32 sum of n terms
            (n u of the sum of magnitudes), half a BF16 step."""
import pytest
import torch

import bit_microscaled_numerics_amd as nv
from parity import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = 2.0 ** -8
CODE = 0.5 * 64 / 65535 * 0.6931472 * 1.001


class Ref:
    """The definitions in binary64, and bounds of the kernels' errors."""

    def __init__(self, h, w, t, weight=None):
        h, w, t = h.cpu().double(), w.cpu().double(), t.cpu().long()
        T, V, D = h.shape[0], w.shape[0], h.shape[1]
        self.live = (t >= 0) & (t < V)
        z = h @ w.t()
        self.dz = (D * U * (h.abs() @ w.abs().t())).amax(1) if T else torch.zeros(0).double()
        self.lse = torch.logsumexp(z, 1)
        at = t.clamp(0, V - 1).unsqueeze(1)
        raw = self.lse - z.gather(1, at).squeeze(1)
        self.loss = torch.where(self.live, raw, torch.zeros_like(raw))
        rel = (80 + V / 128 / 64 + 8) * U + 8 * U
        self.tol_lse = self.dz + rel + U * self.lse.abs()
        self.tol_loss = torch.where(self.live, 2 * self.dz + rel + U * raw.abs(), torch.zeros_like(raw))
        if weight is None:
            weight = torch.full((T,), 1.0 / max(1, int(self.live.sum())))
        g = torch.where(self.live, weight.cpu().double(), torch.zeros(T).double()).unsqueeze(1)
        p = torch.exp(z - self.lse.unsqueeze(1))
        onehot = torch.zeros_like(p).scatter_(1, at, 1.0)
        d = g * (p - onehot)
        ez = (2 * self.dz + rel).unsqueeze(1)
        err = g.abs() * p * (CODE * (1 - onehot) + 2 * ez + 8 * U) + g.abs() * 1e-18
        err = err * (1 + HALF) + HALF * d.abs()
        dead = ~self.live.unsqueeze(1)
        # a row without a target holds anything
        h = torch.where(dead, torch.zeros_like(h), h)
        d, err = torch.where(dead, 0.0, d), torch.where(dead, 0.0, err)
        self.dh, self.dw = d @ w, d.t() @ h
        mag = d.abs() + err
        self.tol_dh = err @ w.abs() + (V + 130) * U * (mag @ w.abs())
        self.tol_dw = err.t() @ h.abs() + (T + 130) * U * (mag.t() @ h.abs())
        self.tol_dh += HALF * (self.dh.abs() + self.tol_dh)
        self.tol_dw += HALF * (self.dw.abs() + self.tol_dw)


def _close(got, ref, tol, what):
    err = (got.cpu().double() - ref).abs()
    bad = torch.nonzero(~(err <= tol))
    assert bad.numel() == 0, (what, len(bad), bad[0].tolist(), err[tuple(bad[0])].item(), tol[tuple(bad[0])].item())


def _inputs(T, V, D, seed=0, ignored="some", scale=0.3, it=torch.int64):
    g = torch.Generator().manual_seed(seed + T * 7 + V * 3 + D)
    h = torch.randn(T, D, generator=g).to(torch.bfloat16)
    w = (torch.randn(V, D, generator=g) * scale).to(torch.bfloat16)
    t = torch.randint(0, V, (T,), generator=g)
    if ignored == "some":
        r = torch.rand(T, generator=g)
        t = torch.where(r < 0.1, torch.full_like(t, -100), torch.where(r < 0.2, t + V, t))
    elif ignored == "all":
        t = torch.full_like(t, -100)
    return h.cuda(), w.cuda(), t.to(it).cuda()


def _check_all(h, w, t, weight=None, piece=0):
    ref = Ref(h, w, t, weight)
    loss, lse = nv.linear_ce(h, w, t)
    _close(loss, ref.loss, ref.tol_loss, "loss")
    _close(lse, ref.lse, ref.tol_lse, "lse")
    loss, lse, dh, dw = nv.linear_ce_grad(h, w, t, row_weight=weight, piece_tokens=piece)
    _close(loss, ref.loss, ref.tol_loss, "loss with gradient")
    _close(lse, ref.lse * ref.live, ref.tol_lse, "lse with gradient")
    _close(dh, ref.dh, ref.tol_dh, "dh")
    _close(dw, ref.dw, ref.tol_dw, "dw")
    return loss, lse, dh, dw


# one token, both sides of the token tiles (64, 128, 256), of a span (128) and
# tile (256) of words, of a step (64) and an instruction (16) of D
@pytest.mark.parametrize("T", [1, 5, 64, 65, 129, 257])
@pytest.mark.parametrize("V", [1, 7, 128, 129, 300, 1027])
@pytest.mark.parametrize("D", [8, 64, 72, 264])
def test_sizes(T, V, D):
    say("ce", T, V, D)
    _check_all(*_inputs(T, V, D, it=torch.int32 if (T + V) % 2 else torch.int64))


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17])
@pytest.mark.parametrize("V,D", [(5, 8), (130, 40), (1000, 256), (4100, 264), (700, 2000)])
@pytest.mark.parametrize("ignored", ["none", "some"])
def test_few_tokens(T, V, D, ignored):
    """Single tokens to a decoding batch, D that is no multiple of a stage (64)."""
    say("ce few", T, V, D, ignored)
    _check_all(*_inputs(T, V, D, scale=0.1, ignored=ignored))


@pytest.mark.parametrize("T,V,D", [(300, 4099, 520), (520, 33000, 136), (40, 9000, 1032)])
@pytest.mark.parametrize("weighted", [False, True])
def test_larger(T, V, D, weighted):
    """Several tiles in each direction, and a dH sum cut into parts."""
    say("ce", T, V, D, weighted)
    h, w, t = _inputs(T, V, D, scale=0.1)
    weight = None
    if weighted:
        weight = torch.rand(T, generator=torch.Generator().manual_seed(1)).sub_(0.2).cuda()
        weight[::5] = 0.0
    _check_all(h, w, t, weight)


@pytest.mark.parametrize("ignored", ["none", "all"])
@pytest.mark.parametrize("T", [1, 70, 300])
def test_masks(T, ignored):
    say("ce mask", T, ignored)
    h, w, t = _inputs(T, 500, 64, ignored=ignored)
    _, _, dh, dw = _check_all(h, w, t)
    if ignored == "all":
        assert torch.all(dh == 0) and torch.all(dw == 0)


def test_no_tokens():
    h, w, t = _inputs(0, 40, 16)
    loss, lse = nv.linear_ce(h, w, t)
    assert loss.shape == (0,) and lse.shape == (0,)
    loss, lse, dh, dw = nv.linear_ce_grad(h, w, t)
    assert loss.shape == (0,) and dh.shape == (0, 16)
    assert torch.all(dw == 0)


@pytest.mark.parametrize("T,piece", [(300, 64), (300, 100), (257, 256), (700, 256)])
@pytest.mark.parametrize("ignored", ["none", "some", "all"])
def test_pieces(T, piece, ignored):
    """dW is added up in FP32 over pieces, the last of them short or empty."""
    say("ce pieces", T, piece, ignored)
    h, w, t = _inputs(T, 777, 136, ignored=ignored)
    if ignored == "some":
        t[T // 3:] = -100   # whole pieces without a token
    _check_all(h, w, t, piece=piece)


def test_strides_and_neighbours():
    """Pitches above the width, outputs inside larger buffers."""
    T, V, D = 77, 333, 72
    h, w, t = _inputs(T, V, D)
    hb = torch.full((T + 1, D + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    wb = torch.full((V + 1, D + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    hv, wv = hb[:T, 8:D + 8], wb[:V, :D]
    hv.copy_(h)
    wv.copy_(w)
    dh = torch.full((T, D + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((V, D + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    ws = torch.empty(nv.nvfp4_linear_ce_workspace_bytes(T, V, D, True), dtype=torch.uint8, device="cuda")
    say("ce strides")
    nv.nvfp4_linear_ce_grad(hv, wv, t, None, 0, loss, lse, dh[:, :D], dw[:, 8:], ws)
    ref = Ref(h, w, t)
    _close(loss, ref.loss, ref.tol_loss, "loss")
    _close(dh[:, :D], ref.dh, ref.tol_dh, "dh")
    _close(dw[:, 8:], ref.dw, ref.tol_dw, "dw")
    assert torch.all(dh[:, D:] == 5.0) and torch.all(dw[:, :8] == 5.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite_rows_without_a_target_reach_nothing(bad):
    h, w, t = _inputs(100, 300, 64, ignored="none")
    t[10:20] = -100
    want = nv.linear_ce_grad(h, w, t)
    h[10:20] = bad
    got = nv.linear_ce_grad(h, w, t)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite_rows_with_a_target_show(bad):
    h, w, t = _inputs(100, 300, 64, ignored="none")
    want_loss, want_lse, want_dh, _ = nv.linear_ce_grad(h, w, t)
    h[33, 5] = bad
    loss, lse, dh, dw = nv.linear_ce_grad(h, w, t)
    assert not torch.isfinite(loss[33]) and not torch.isfinite(dh[33]).any()
    keep = torch.arange(100, device="cuda") != 33
    assert torch.equal(loss[keep], want_loss[keep]) and torch.equal(dh[keep], want_dh[keep])


@pytest.mark.parametrize("scale", [8.0, 60.0])
def test_large_logits(scale):
    """Logits in the hundreds and thousands: nearly all of the mass on one word,
    most exponentials 0, losses near 0 and large ones side by side."""
    h, w, t = _inputs(140, 400, 64, ignored="none", scale=scale)
    best = (h.float() @ w.float().t()).argmax(1)
    t[::2] = best[::2]
    _check_all(h, w, t)


def test_one_word_and_equal_logits():
    h = torch.zeros(9, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1000, 16, dtype=torch.bfloat16, device="cuda")
    t = torch.arange(9, device="cuda")
    _check_all(h, w, t)


def test_gradient_against_differences():
    """The directional derivative of the weighted loss, by central differences of
    the binary64 definition, against the kernels' gradient along the same
    direction (step 1e-4: error 1e-8 of the third derivative)."""
    T, V, D = 60, 200, 48
    h, w, t = _inputs(T, V, D)
    weight = torch.rand(T, generator=torch.Generator().manual_seed(2)).cuda()
    ref = Ref(h, w, t, weight)
    _, _, dh, dw = nv.linear_ce_grad(h, w, t, row_weight=weight)
    g = torch.Generator().manual_seed(3)
    uh, uw = torch.randn(T, D, generator=g).double(), torch.randn(V, D, generator=g).double()

    def value(eps):
        r = (h.cpu().double() + eps * uh) @ (w.cpu().double() + eps * uw).t()
        tt = t.cpu()
        raw = torch.logsumexp(r, 1) - r.gather(1, tt.clamp(0, V - 1).unsqueeze(1)).squeeze(1)
        return (raw * weight.cpu().double())[ref.live].sum()

    slope = (value(1e-4) - value(-1e-4)) / 2e-4
    got = (dh.cpu().double() * uh).sum() + (dw.cpu().double() * uw).sum()
    tol = (ref.tol_dh * uh.abs()).sum() + (ref.tol_dw * uw.abs()).sum() + 1e-4 * slope.abs()
    assert abs(got - slope) <= tol


def test_same_bits_every_time():
    h, w, t = _inputs(600, 9001, 200)
    first = nv.linear_ce_grad(h, w, t)
    for _ in range(3):
        for a, b in zip(nv.linear_ce_grad(h, w, t), first):
            assert torch.equal(a, b)


def test_on_another_stream_and_in_a_graph():
    T, V, D = 200, 1500, 96
    h, w, t = _inputs(T, V, D)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    ws = torch.empty(nv.nvfp4_linear_ce_workspace_bytes(T, V, D, True), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    nv.nvfp4_linear_ce_grad(h, w, t, None, 0, loss, lse, dh, dw, ws, stream=side)
    side.synchronize()
    ref = Ref(h, w, t)
    _close(dw, ref.dw, ref.tol_dw, "dw")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_linear_ce_grad(h, w, t, None, 0, loss, lse, dh, dw, ws)
    for seed in range(3):
        h2, _, t2 = _inputs(T, V, D, seed=seed + 1, ignored="none" if seed == 1 else "some")
        h.copy_(h2)
        t.copy_(t2)
        for x in (loss, lse, dh, dw):
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((loss, lse, dh, dw), nv.linear_ce_grad(h, w, t)):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """A vocabulary matrix of 5.2 GB: the last words' logits and gradients."""
    T, V, D = 8, 320000, 8192
    say("ce 5.2 GB", T, V, D)
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(V, D, dtype=torch.bfloat16, device="cuda").normal_(0, 0.01, generator=g)
    h = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    t = V - 1 - torch.arange(T, device="cuda") * 40000
    loss, _, dh, dw = nv.linear_ce_grad(h, w, t)
    z = torch.cat([h.double() @ w[v:v + 16000].double().t() for v in range(0, V, 16000)], 1)
    p = torch.softmax(z, 1)
    p[torch.arange(T), t] -= 1
    ref = torch.logsumexp(z, 1) - z.gather(1, t.unsqueeze(1)).squeeze(1)
    # |h w| sums to about 0.0064 D = 52: dz = D u 52 = 0.026 is the worst case; rounding errors of
    # random sign grow as sqrt(D): 3e-4
    assert torch.all((loss.double() - ref).abs() <= 0.026 * 2)
    p /= T
    d_dh = sum(p[:, v:v + 16000] @ w[v:v + 16000].double() for v in range(0, V, 16000))
    assert (dh.double() - d_dh).norm() <= (2 * HALF + 0.052) * d_dh.norm()
    last = p[:, V - 300:].t() @ h.double()
    assert (dw[V - 300:].double() - last).norm() <= (2 * HALF + 0.052) * last.norm()


@pytest.mark.parametrize("V,D", [(100003, 2568), (131072, 2056)])
def test_long_products(V, D):
    """8192 tokens and enough words that each workgroup takes thousands of steps, of
    which the parts of a product differ in length.  64 distinct tokens, repeated with
    weights of their own, keep the reference small."""
    say("ce long", V, D)
    U64, T = 64, 8192
    hu, w, tu = _inputs(U64, V, D, ignored="none", scale=0.05)
    rep = torch.arange(T, device="cuda") % U64
    g = torch.Generator().manual_seed(V)
    weight = torch.rand(T, generator=g).cuda()
    weight[weight < 0.05] = 0.0
    h, t = hu[rep].contiguous(), tu[rep].contiguous()
    loss, lse, dh, dw = nv.linear_ce_grad(h, w, t, row_weight=weight)
    again = nv.linear_ce_grad(h, w, t, row_weight=weight)
    assert torch.equal(dh, again[2]) and torch.equal(dw, again[3])

    h64, w64 = hu.double(), w.double()
    z = torch.empty(U64, V, dtype=torch.float64, device="cuda")
    mag_z = 0.0
    for v in range(0, V, 8192):
        part = w64[v:v + 8192].t().contiguous()
        z[:, v:v + 8192] = h64 @ part
        mag_z = max(mag_z, float((h64.abs() @ part.abs()).max()))
    ref_lse = torch.logsumexp(z, 1)
    at = tu.long().unsqueeze(1)
    ref_loss = ref_lse - z.gather(1, at).squeeze(1)
    dz, rel = D * U * mag_z, (80 + V / 128 / 64 + 8) * U + 8 * U
    assert ((lse.double() - ref_lse[rep]).abs() <= dz + rel + U * ref_lse[rep].abs()).all()
    assert ((loss.double() - ref_loss[rep]).abs() <= 2 * dz + rel + U * ref_loss[rep].abs()).all()
    p = torch.exp(z - ref_lse.unsqueeze(1))
    onehot = torch.zeros_like(p).scatter_(1, at, 1.0)
    d = p - onehot
    err = p * (CODE * (1 - onehot) + 2 * (2 * dz + rel) + 8 * U) + 1e-18
    # weights are held relative to their largest: one more rounding of u each way
    err = err * (1 + HALF) + (HALF + 3 * U) * d.abs()
    each = weight.double().unsqueeze(1)
    total = torch.zeros(U64, 1, dtype=torch.float64, device="cuda").index_add_(0, rep, each)
    dh_u = tol_dh_u = 0.0
    h_abs = h64.abs()
    for v in range(0, V, 8192):
        part, s = w64[v:v + 8192], slice(v, v + 8192)
        dh_u = dh_u + d[:, s] @ part
        e, m = err[:, s].contiguous(), (d[:, s].abs() + err[:, s])
        tol_dh_u = tol_dh_u + e @ part.abs() + (V + 130) * U * (m @ part.abs())
        ref = (total * d[:, s]).t().contiguous() @ h64
        tol = (total * e).t().contiguous() @ h_abs + (T + 130) * U * ((total * m).t().contiguous() @ h_abs)
        tol = tol + HALF * (ref.abs() + tol)
        off = (dw[s].double() - ref).abs()
        assert (off <= tol).all(), ("dw", v, (off - tol).max().item())
    for i in range(0, T, U64):
        ref, tol = each[i:i + U64] * dh_u, each[i:i + U64] * tol_dh_u
        off = (dh[i:i + U64].double() - ref).abs()
        assert (off <= tol + HALF * (ref.abs() + tol)).all(), ("dh", i)


@pytest.mark.parametrize("T", [1, 16, 31, 32, 33])
@pytest.mark.parametrize("V,D", [(1, 8), (63, 136), (1025, 72), (2111, 1000)])
@pytest.mark.parametrize("ignored", ["none", "some", "all"])
def test_few_tokens_and_their_words(T, V, D, ignored):
    """Both sides of the kernel for few tokens; odd vocabularies and widths."""
    say("ce few", T, V, D, ignored)
    h, w, t = _inputs(T, V, D, seed=3, ignored=ignored)
    g = torch.Generator().manual_seed(T)
    weight = torch.rand(T, generator=g) * torch.randint(0, 2, (T,), generator=g)
    _, _, dh, dw = _check_all(h, w, t)
    if ignored == "all":
        assert not dh.any() and not dw.any()
    # results inside a wider matrix: nothing is written beside them
    wide = torch.full((V, D + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    ws = torch.empty(nv.nvfp4_linear_ce_workspace_bytes(T, V, D, True), dtype=torch.uint8, device="cuda")
    nv.nvfp4_linear_ce_grad(h, w, t, weight.cuda(), 0, loss, lse, dh, wide[:, :D], ws)
    ref = Ref(h, w, t, weight)
    _close(wide[:, :D], ref.dw, ref.tol_dw + 3 * U * ref.dw.abs(), "dw")
    assert torch.all(wide[:, D:] == 3.0)


def test_more_tokens_than_a_launch_has_threads():
    """2^26 tokens and some: one wave each is 2^32 threads, more than one dimension of
    a launch holds.  The first and the last tokens have targets."""
    T, V, D, U64 = (1 << 26) + 71, 5, 8, 64
    say("ce 2^26", T)
    hu, w, tu = _inputs(U64, V, D, ignored="none")
    rep = torch.arange(T, device="cuda", dtype=torch.int32) % U64
    h, t = hu.repeat(T // U64 + 1, 1)[:T], tu.repeat(T // U64 + 1)[:T]   # row i is hu[rep[i]]
    ref = Ref(hu, w, tu)
    loss, lse = nv.linear_ce(h, w, t)
    for s in (slice(0, 1 << 20), slice(T - (1 << 20), T), slice((1 << 26) - 512, T)):
        r = rep[s].cpu().long()
        _close(loss[s], ref.loss[r], ref.tol_loss[r], "loss")
        _close(lse[s], ref.lse[r], ref.tol_lse[r], "lse")
    cut = 500   # live tokens at either end
    t[cut:T - cut] = -100
    loss, lse, dh, dw = nv.linear_ce_grad(h, w, t)
    ends = torch.cat([torch.arange(cut), torch.arange(T - cut, T)]).cuda()
    ref = Ref(h[ends], w, t[ends])
    _close(loss[ends], ref.loss, ref.tol_loss, "loss with gradient")
    _close(dh[ends], ref.dh, ref.tol_dh, "dh")
    _close(dw, ref.dw, ref.tol_dw, "dw")
    assert not loss[cut:T - cut].any() and not dh[cut:T - cut].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T", [20, 100])
def test_nonfinite_rows_of_weight_zero_reach_no_gradient(T, bad):
    """A weight of 0 masks a token: what its row holds stays out of dh and dw."""
    say("ce weight 0", T, bad)
    h, w, t = _inputs(T, 300, 64, ignored="none")
    weight = torch.rand(T, generator=torch.Generator().manual_seed(4)).cuda()
    weight[5:9] = 0.0
    weight[11] = -0.0
    want = nv.linear_ce_grad(h, w, t, row_weight=weight)
    h[5:9], h[11] = bad, bad
    for piece in (0, 16):
        loss, lse, dh, dw = nv.linear_ce_grad(h, w, t, row_weight=weight, piece_tokens=piece)
        keep = weight != 0
        assert torch.equal(loss[keep], want[0][keep]) and not torch.isfinite(loss[~keep]).any()
        assert torch.equal(dh, want[2]) and torch.all(dh[~keep] == 0)
        if piece == 0:
            assert torch.equal(dw, want[3])
        else:
            ref = Ref(torch.where(keep.unsqueeze(1), h, torch.zeros_like(h)), w, t, weight)
            _close(dw, ref.dw, ref.tol_dw, "dw in pieces")


@pytest.mark.parametrize("V", [300, 4099])
def test_confident_tokens(V):
    """Targets that lead by 1 .. 60 in the logit: the losses of the surest are below what
    binary32 sums near 1 can show, and still not negative, nor does the gradient push a
    target away; within the bounds above."""
    T, D = 60, 64
    say("ce confident", V)
    g = torch.Generator().manual_seed(V)
    w = (torch.randn(V, D, generator=g) * 0.01).to(torch.bfloat16)
    t = torch.randperm(V, generator=g)[:T]
    h = torch.randn(T, D, generator=g).to(torch.bfloat16)
    for i in range(T):   # the words of the targets point along their rows
        hi = h[i].float()
        w[t[i]] = (hi * ((i + 1.0) / (hi @ hi))).to(torch.bfloat16)
    h, w, t = h.cuda(), w.cuda(), t.cuda()
    assert Ref(h, w, t).loss.min() < 1e-9
    loss, _, _, _ = _check_all(h, w, t)
    assert torch.all(loss >= 0) and torch.all(nv.linear_ce(h, w, t)[0] >= 0)
    one = torch.ones(T, device="cuda")
    for i in range(T - 8, T):   # one live row at a time: its target's row of dw is d h, d <= 0
        alone = torch.full_like(t, -100)
        alone[i] = t[i]
        _, _, _, dw = nv.linear_ce_grad(h, w, alone, row_weight=one)
        assert torch.all(dw[t[i]].float() * h[i].float() <= 0)


def test_widest_rows():
    """D just below 2^22 with a whole tile of tokens: the gathered rows' byte offsets
    stay below 2^31.  Everything else in the workspace starts as NaN."""
    T, V, D = 257, 3, (1 << 22) - 8
    say("ce wide", T, V, D)
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    w = torch.empty(V, D, dtype=torch.bfloat16, device="cuda").normal_(0, 0.0005, generator=g)
    t = torch.arange(T, device="cuda") % V
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    ws = torch.full((nv.nvfp4_linear_ce_workspace_bytes(T, V, D, True),), 255, dtype=torch.uint8,
                    device="cuda")
    nv.nvfp4_linear_ce_grad(h, w, t, None, 0, loss, lse, dh, dw, ws)
    z = torch.zeros(T, V, dtype=torch.float64, device="cuda")
    for c in range(0, D, 1 << 18):
        z += h[:, c:c + (1 << 18)].double() @ w[:, c:c + (1 << 18)].double().t().contiguous()
    p = torch.softmax(z, 1)
    p[torch.arange(T), t] -= 1
    ref = torch.logsumexp(z, 1) - z.gather(1, t.unsqueeze(1)).squeeze(1)
    # partial sums are of the order 0.0005 sqrt(D) = 1: D / 16 roundings of u each are at
    # most 0.016 in z, relative in p
    assert torch.all((loss.double() - ref).abs() <= 0.032)
    p /= T
    for c in (0, 1 << 21, D - 4096):
        s = slice(c, c + 4096)
        rdh = p @ w[:, s].double()
        rdw = p.t().contiguous() @ h[:, s].double()
        assert (dh[:, s].double() - rdh).norm() <= (2 * HALF + 0.032) * rdh.norm()
        assert (dw[:, s].double() - rdw).norm() <= (2 * HALF + 0.032) * rdw.norm()


def _check_repeated(hu, w, tu, rep, weight, piece):
    """Token i is row rep[i] of the distinct ones (hu, tu), with a weight of its own: the
    reference needs only the distinct rows' logits.  Bounds as above; weights are held
    relative to their largest, one more rounding of u each way.  In blocks of words, so that
    w may pass 2^32 bytes."""
    distinct, (V, D), T = hu.shape[0], w.shape, rep.numel()
    h, t = hu[rep].contiguous(), tu[rep].contiguous()
    loss, lse, dh, dw = nv.linear_ce_grad(h, w, t, row_weight=weight, piece_tokens=piece)
    again = nv.linear_ce_grad(h, w, t, row_weight=weight, piece_tokens=piece)
    assert torch.equal(dh, again[2]) and torch.equal(dw, again[3])
    del again
    live = (tu >= 0) & (tu < V)
    h64 = hu.double()
    z = torch.empty(distinct, V, dtype=torch.float64, device="cuda")
    dz = torch.zeros(distinct, dtype=torch.float64, device="cuda")
    for v in range(0, V, 8192):
        part = w[v:v + 8192].double().t().contiguous()
        z[:, v:v + 8192] = h64 @ part
        dz = torch.maximum(dz, (h64.abs() @ part.abs()).amax(1))
    dz, rel = D * U * dz, (80 + V / 128 / 64 + 8) * U + 8 * U
    ref_lse = torch.logsumexp(z, 1)
    at = tu.long().clamp(0, V - 1).unsqueeze(1)
    ref_loss = (ref_lse - z.gather(1, at).squeeze(1)) * live
    ok = (loss.double() - ref_loss[rep]).abs() <= (2 * dz + rel + U * ref_loss)[rep] * live[rep]
    assert ok.all(), "loss"
    ok = (lse.double() - (ref_lse * live)[rep]).abs() <= (dz + rel + U * ref_lse.abs())[rep] * live[rep]
    assert ok.all(), "lse"
    p = torch.exp(z - ref_lse.unsqueeze(1)) * live.unsqueeze(1)
    onehot = torch.zeros_like(p).scatter_(1, at, 1.0) * live.unsqueeze(1)
    d = p - onehot
    err = p * (CODE * (1 - onehot) + 2 * (2 * dz + rel).unsqueeze(1) + 8 * U) + 1e-18 * live.unsqueeze(1)
    err = err * (1 + HALF) + (HALF + 3 * U) * d.abs()
    each = weight.double().unsqueeze(1)
    total = torch.zeros(distinct, 1, dtype=torch.float64, device="cuda").index_add_(0, rep, each)
    dh_u = tol_u = 0.0
    for v in range(0, V, 8192):
        part, s = w[v:v + 8192].double(), slice(v, v + 8192)
        e, m = err[:, s].contiguous(), d[:, s].abs() + err[:, s]
        dh_u = dh_u + d[:, s].contiguous() @ part
        tol_u = tol_u + e @ part.abs() + (V + 130) * U * (m @ part.abs())
        ref = (total * d[:, s]).t().contiguous() @ h64
        tol = (total * e).t().contiguous() @ h64.abs()
        tol = tol + (T + 130) * U * ((total * m).t().contiguous() @ h64.abs())
        off = (dw[s].double() - ref).abs()
        assert (off <= tol + HALF * (ref.abs() + tol)).all(), ("dw", v)
    for i in range(0, T, 4096):
        r = rep[i:i + 4096]
        ref, tol = each[i:i + 4096] * dh_u[r], each[i:i + 4096] * tol_u[r]
        off = (dh[i:i + 4096].double() - ref).abs()
        assert (off <= tol + HALF * (ref.abs() + tol)).all(), ("dh", i)


@pytest.mark.parametrize("T,D,piece", [(16484, 2056, 8192), (16484, 2056, 0), (16484, 1032, 5000)])
def test_long_pieces(T, D, piece):
    """Long products in pieces: dW's sums go on in FP32 from piece to piece, the workgroups
    kept together (2048 steps and more) in the whole pieces and not in the short last one.
    piece 0: the 4 GiB of codes for 131072 words hold 16128 tokens, so the default has two
    pieces too.  Tokens without a target and of weight 0 among them."""
    V, distinct = 131072, 64
    say("ce long pieces", T, D, piece)
    hu, w, tu = _inputs(distinct, V, D, ignored="none", scale=0.05)
    tu[5::16] = -100
    rep = torch.arange(T, device="cuda") * 7 % distinct
    weight = torch.rand(T, generator=torch.Generator().manual_seed(D + piece)).cuda()
    weight[weight < 0.05] = 0.0
    _check_repeated(hu, w, tu, rep, weight, piece)


@pytest.mark.parametrize("T", [33, 130])
def test_words_gradient_past_32_bits(T):
    """dW of 5.2 GB from the general kernel (more than 32 tokens)."""
    V, D = 320000, 8192
    say("ce dw 5.2 GB", T)
    g = torch.Generator(device="cuda").manual_seed(T)
    w = torch.empty(V, D, dtype=torch.bfloat16, device="cuda").normal_(0, 0.01, generator=g)
    h = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    t = V - 1 - torch.arange(T, device="cuda") * 2400
    weight = torch.rand(T, generator=g, device="cuda")
    _check_repeated(h, w, t, torch.arange(T, device="cuda"), weight, 0)
