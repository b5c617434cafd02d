"""Refusals of the embedding, gradient-clipping and cross-entropy entry points: bad
arguments are named before anything is enqueued, in the C ABI and in the
binding.  CPU only."""
import ctypes

import pytest
import torch

import bit_microscaled_numerics_amd as nv

FAKE, MIS = 0x10000, 0x10001
BF, F, I4, I8 = nv.NVFP4_TYPE_BF16, nv.NVFP4_TYPE_F32, nv.NVFP4_TYPE_I32, nv.NVFP4_TYPE_I64


@pytest.fixture(scope="module")
def lib():
    return nv.load_library()


def _embed(lib, ids=FAKE, it=I8, n=4, w=FAKE, wt=BF, V=10, D=7, ldw=7, out=FAKE, ot=F, ldo=7):
    return lib.nvfp4_embed(ids, it, n, w, wt, V, D, ldw, 1.0, out, ot, ldo, None)


@pytest.mark.parametrize("kw,status", [
    (dict(ids=None), nv.NVFP4_ERR_NULL), (dict(w=None), nv.NVFP4_ERR_NULL),
    (dict(out=None), nv.NVFP4_ERR_NULL), (dict(n=-1), nv.NVFP4_ERR_SHAPE),
    (dict(n=1 << 31), nv.NVFP4_ERR_SHAPE), (dict(V=0), nv.NVFP4_ERR_SHAPE),
    (dict(V=(1 << 31) - 1), nv.NVFP4_ERR_SHAPE), (dict(D=0), nv.NVFP4_ERR_SHAPE),
    (dict(D=(1 << 24) + 1, ldw=1 << 25, ldo=1 << 25), nv.NVFP4_ERR_SHAPE),
    (dict(ldw=6), nv.NVFP4_ERR_SHAPE), (dict(ldo=6), nv.NVFP4_ERR_SHAPE),
    (dict(ldw=1 << 38), nv.NVFP4_ERR_SHAPE), (dict(it=BF), nv.NVFP4_ERR_ARG),
    (dict(wt=I4), nv.NVFP4_ERR_ARG), (dict(ot=9), nv.NVFP4_ERR_ARG),
    (dict(ids=MIS), nv.NVFP4_ERR_ALIGN), (dict(w=MIS), nv.NVFP4_ERR_ALIGN),
    (dict(out=FAKE + 2), nv.NVFP4_ERR_ALIGN)])
def test_embed_validation(lib, kw, status):
    assert _embed(lib, **kw) == status
    assert lib.nvfp4_last_error()


def _embed_grad(lib, ids=FAKE, it=I4, n=4, dy=FAKE, yt=F, ldy=7, V=10, D=7, dw=FAKE, wt=F, ldw=7,
                acc=0, ws=FAKE, nb=1 << 20):
    return lib.nvfp4_embed_grad(ids, it, n, dy, yt, ldy, V, D, 1.0, dw, wt, ldw, acc, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(ids=None), nv.NVFP4_ERR_NULL), (dict(dy=None), nv.NVFP4_ERR_NULL),
    (dict(dw=None), nv.NVFP4_ERR_NULL), (dict(ws=None), nv.NVFP4_ERR_NULL),
    (dict(n=-5), nv.NVFP4_ERR_SHAPE), (dict(V=-1), nv.NVFP4_ERR_SHAPE),
    (dict(ldy=3), nv.NVFP4_ERR_SHAPE), (dict(ldw=3), nv.NVFP4_ERR_SHAPE),
    (dict(it=F), nv.NVFP4_ERR_ARG), (dict(yt=I8), nv.NVFP4_ERR_ARG),
    (dict(wt=I8), nv.NVFP4_ERR_ARG), (dict(acc=2), nv.NVFP4_ERR_ARG),
    (dict(nb=8), nv.NVFP4_ERR_ARG), (dict(ws=FAKE + 16), nv.NVFP4_ERR_ALIGN),
    (dict(ids=FAKE + 2), nv.NVFP4_ERR_ALIGN), (dict(dy=FAKE + 2), nv.NVFP4_ERR_ALIGN)])
def test_embed_grad_validation(lib, kw, status):
    assert _embed_grad(lib, **kw) == status


def test_embed_grad_workspace_query(lib):
    q = lib.nvfp4_embed_grad_workspace_bytes
    assert q(0, 10, 8) == 0
    assert q(-1, 10, 8) == nv.NVFP4_ERR_SHAPE and q(4, 0, 8) == nv.NVFP4_ERR_SHAPE
    assert 0 < q(8192, 131072, 5120) < 1 << 23
    assert q(16385, 10, 8) > q(16384, 10, 8) > 0
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_embed_grad_workspace_bytes(4, 10, 0)


def _grads(*rows):
    arr = (nv.c_grad * len(rows))()
    for a, r in zip(arr, rows):
        a.in_, a.out, a.numel, a.in_type, a.out_type = r
    return arr


@pytest.mark.parametrize("row,status", [
    ((None, FAKE, 4, F, F), nv.NVFP4_ERR_NULL), ((FAKE, None, 4, F, F), nv.NVFP4_ERR_NULL),
    ((FAKE, FAKE, -4, F, F), nv.NVFP4_ERR_SHAPE), ((FAKE, FAKE, (1 << 40) + 1, F, F), nv.NVFP4_ERR_SHAPE),
    ((FAKE, FAKE + 64, 4, I4, F), nv.NVFP4_ERR_ARG), ((FAKE, FAKE + 64, 4, F, I8), nv.NVFP4_ERR_ARG),
    ((FAKE, FAKE, 4, F, BF), nv.NVFP4_ERR_ARG), ((FAKE + 2, FAKE, 4, F, F), nv.NVFP4_ERR_ALIGN),
    ((FAKE, MIS, 4, BF, BF), nv.NVFP4_ERR_ALIGN)])
def test_clip_list_validation(lib, row, status):
    good = (FAKE, FAKE, 4, F, F)
    lst = ctypes.cast(_grads(good, row), ctypes.c_void_p)
    assert lib.nvfp4_grad_clip(lst, 2, FAKE, 1.0, FAKE, None) == status
    assert b"gradient 1" in lib.nvfp4_last_error()


def test_clip_argument_validation(lib):
    lst = ctypes.cast(_grads((FAKE, FAKE, 4, F, F)), ctypes.c_void_p)
    c = lib.nvfp4_grad_clip
    assert c(lst, -1, FAKE, 1.0, FAKE, None) == nv.NVFP4_ERR_SHAPE
    assert c(None, 1, FAKE, 1.0, FAKE, None) == nv.NVFP4_ERR_NULL
    assert c(lst, 1, None, 1.0, FAKE, None) == nv.NVFP4_ERR_NULL
    assert c(lst, 1, FAKE + 4, 1.0, FAKE, None) == nv.NVFP4_ERR_ALIGN
    assert c(lst, 1, FAKE, -1.0, FAKE, None) == nv.NVFP4_ERR_ARG
    assert c(lst, 1, FAKE, float("nan"), FAKE, None) == nv.NVFP4_ERR_ARG
    assert c(lst, 1, FAKE, 1.0, FAKE + 2, None) == nv.NVFP4_ERR_ALIGN
    assert lib.nvfp4_grad_sumsq(lst, 1, None, None) == nv.NVFP4_ERR_NULL
    assert lib.nvfp4_grad_sumsq(None, 1, FAKE, None) == nv.NVFP4_ERR_NULL


def test_scale_argument_validation(lib):
    lst = ctypes.cast(_grads((FAKE, FAKE, 4, F, F)), ctypes.c_void_p)
    assert lib.nvfp4_grad_scale(lst, 1, None, None) == nv.NVFP4_ERR_NULL
    assert lib.nvfp4_grad_scale(lst, 1, FAKE + 2, None) == nv.NVFP4_ERR_ALIGN
    assert lib.nvfp4_grad_scale(lst, -1, FAKE, None) == nv.NVFP4_ERR_SHAPE
    assert lib.nvfp4_grad_scale(None, 1, FAKE, None) == nv.NVFP4_ERR_NULL


def test_binding_refuses():
    ids = torch.zeros(4, dtype=torch.int64)
    w = torch.zeros(8, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        nv.embed(ids, w)
    with pytest.raises(ValueError, match="CUDA"):
        nv.embed_grad(ids, w[:4], 8)
    with pytest.raises(ValueError, match="CUDA"):
        nv.clip_grads([w], 1.0)
    with pytest.raises(ValueError, match="at least one"):
        nv.clip_grads([], 1.0)
    with pytest.raises(ValueError, match="one output"):
        nv.clip_grads([w, w], 1.0, out=[w])
    with pytest.raises(ValueError, match="no gradients"):
        nv.grad_sumsq([])
    with pytest.raises(ValueError, match="overlapping"):
        nv._pitch(torch.zeros(1, 4).expand(3, 4), "x")
    assert nv._pitch(torch.zeros(1, 4).expand(1, 4), "x") == 4
    assert nv._pitch(torch.zeros(3, 9)[:, :4], "x") == 9


def _ce(lib, grad=True, h=FAKE, ldh=64, w=FAKE, ldw=64, T=4, V=10, D=64, t=FAKE, tt=I8, rw=None,
        piece=0, loss=FAKE, lse=FAKE, dh=FAKE, ld_dh=64, dw=FAKE, ld_dw=64, ws=FAKE, nb=1 << 40):
    if not grad:
        return lib.nvfp4_linear_ce(h, ldh, w, ldw, T, V, D, t, tt, loss, lse, ws, nb, None)
    return lib.nvfp4_linear_ce_grad(h, ldh, w, ldw, T, V, D, t, tt, rw, piece, loss, lse, dh, ld_dh,
                                    dw, ld_dw, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(h=None), nv.NVFP4_ERR_NULL), (dict(w=None), nv.NVFP4_ERR_NULL),
    (dict(t=None), nv.NVFP4_ERR_NULL), (dict(loss=None), nv.NVFP4_ERR_NULL),
    (dict(ws=None), nv.NVFP4_ERR_NULL), (dict(T=-1), nv.NVFP4_ERR_SHAPE),
    (dict(T=(1 << 31) - 1), nv.NVFP4_ERR_SHAPE), (dict(V=0), nv.NVFP4_ERR_SHAPE),
    (dict(V=1 << 31), nv.NVFP4_ERR_SHAPE), (dict(D=0), nv.NVFP4_ERR_SHAPE),
    (dict(D=60), nv.NVFP4_ERR_SHAPE), (dict(ldh=56), nv.NVFP4_ERR_SHAPE),
    (dict(ldw=56), nv.NVFP4_ERR_SHAPE), (dict(ldw=1 << 22), nv.NVFP4_ERR_SHAPE),
    (dict(ldh=68), nv.NVFP4_ERR_ALIGN), (dict(w=FAKE + 8), nv.NVFP4_ERR_ALIGN),
    (dict(lse=FAKE + 2), nv.NVFP4_ERR_ALIGN), (dict(t=FAKE + 4), nv.NVFP4_ERR_ALIGN),
    (dict(ws=FAKE + 128), nv.NVFP4_ERR_ALIGN), (dict(tt=BF), nv.NVFP4_ERR_ARG),
    (dict(nb=64), nv.NVFP4_ERR_ARG), (dict(nb=-1), nv.NVFP4_ERR_ARG)])
@pytest.mark.parametrize("grad", [False, True])
def test_ce_validation(lib, kw, status, grad):
    assert _ce(lib, grad=grad, **kw) == status
    assert lib.nvfp4_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dh=None), nv.NVFP4_ERR_NULL), (dict(dw=None), nv.NVFP4_ERR_NULL),
    (dict(V=1 << 22), nv.NVFP4_ERR_SHAPE), (dict(piece=-1), nv.NVFP4_ERR_SHAPE),
    (dict(ld_dh=8), nv.NVFP4_ERR_SHAPE), (dict(ld_dw=70), nv.NVFP4_ERR_ALIGN),
    (dict(dh=FAKE + 2), nv.NVFP4_ERR_ALIGN), (dict(rw=FAKE + 2), nv.NVFP4_ERR_ALIGN)])
def test_ce_grad_validation(lib, kw, status):
    assert _ce(lib, **kw) == status


def test_ce_workspace_query(lib):
    q = lib.nvfp4_linear_ce_workspace_bytes
    for T in (0, 1, 63, 64, 65, 1000, 100000):
        for V in (1, 127, 50257, 131072):
            small = [q(T, V, D, g, 0) for D in (8, 5120) for g in (0, 1)]
            assert all(0 < b < 1 << 36 for b in small), (T, V, small)
            assert q(T, V, 512, 1, 256) <= q(T, V, 512, 1, 0) + (V + 256) * 512 * 4 + (1 << 20)
    assert q(4, 10, 64, 2, 0) == nv.NVFP4_ERR_ARG
    assert q(4, 10, 63, 1, 0) == nv.NVFP4_ERR_SHAPE
    assert q(-4, 10, 64, 1, 0) == nv.NVFP4_ERR_SHAPE
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_linear_ce_workspace_bytes(4, 0, 64, True)


def test_ce_binding_refuses():
    h = torch.zeros(4, 16, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    for f in (nv.linear_ce, nv.linear_ce_grad):
        with pytest.raises(ValueError, match="CUDA"):
            f(h, h, t)


def test_ce_gathered_rows_stay_below_2_31_bytes(lib):
    """256 gathered rows are one operand with 32-bit byte offsets: their pitch, seen in the
    workspace of one more row, is at most 2^22 elements for every D that is accepted."""
    q = lib.nvfp4_linear_ce_workspace_bytes
    base, at = (1 << 22) - 136, (1 << 22) - 128    # the pitch of rows of `base` elements
    for D in ((1 << 22) - 128, (1 << 22) - 64, (1 << 22) - 8):
        more = q(256, 8, D, 1, 0) - q(256, 8, base, 1, 0)
        assert at + more / 512 <= 1 << 22, D


def test_lists_of_different_lengths_are_refused():
    """Before anything of either list is looked at, from sequences and generators."""
    x, partials, one = torch.zeros(4), torch.zeros(nv.NVFP4_SUMSQ_WORDS), torch.zeros(1)
    for n, m in ((2, 1), (1, 2), (1, 0), (0, 1)):
        for kind in (list, iter):
            with pytest.raises(ValueError, match=f"{m} outputs for {n} gradients"):
                nv.nvfp4_grad_clip(kind([x] * n), kind([x] * m), partials, 1.0, one)
            with pytest.raises(ValueError, match=f"{m} outputs for {n} gradients"):
                nv.nvfp4_grad_scale(kind([x] * n), kind([x] * m), one)


class _Elsewhere:
    """What the checks see of a float32 value (or float64 partial sums) on GPU `device`."""
    is_cuda = True

    def __init__(self, device, n=1, dtype=torch.float32):
        self.device_index, self.n, self.dtype = device, n, dtype

    def is_contiguous(self):
        return True

    def numel(self):
        return self.n

    def get_device(self):
        return self.device_index


def test_norm_and_factor_are_one_float32_on_the_current_device(monkeypatch):
    partials = torch.zeros(nv.NVFP4_SUMSQ_WORDS, dtype=torch.float64)
    for bad in (torch.zeros(1), torch.zeros(1, dtype=torch.bfloat16), torch.zeros(2),
                _Elsewhere(0, n=2), _Elsewhere(0, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="norm_out"):
            nv.nvfp4_grad_clip([], [], partials, 1.0, bad)
        with pytest.raises(ValueError, match="factor"):
            nv.nvfp4_grad_scale([], [], bad)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current CUDA device"):
        nv.nvfp4_grad_clip([], [], partials, 1.0, _Elsewhere(1))
    with pytest.raises(ValueError, match="current CUDA device"):
        nv.nvfp4_grad_scale([], [], _Elsewhere(1))


def test_workspace_is_one_piece():
    """Its size counts from its first byte on: gaps in it belong to somebody else."""
    assert nv._nbytes(None) == 0 and nv._nbytes(torch.zeros(6, dtype=torch.int32)) == 24
    for ws in (torch.zeros(64, dtype=torch.uint8)[::2], torch.zeros(1, dtype=torch.uint8).expand(512),
               torch.zeros(8, 16, dtype=torch.uint8)[:, :8]):
        with pytest.raises(ValueError, match="contiguous"):
            nv._nbytes(ws)


def test_scale_of_a_gradient_without_a_dimension_reaches_its_checks():
    with pytest.raises(ValueError, match="CUDA"):
        nv.scale_grads([torch.tensor(3.0)], torch.ones(1))
