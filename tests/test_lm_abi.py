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
