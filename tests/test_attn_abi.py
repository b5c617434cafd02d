"""Refusals of the query / key norm and rotation and of attention: bad arguments are
named before anything is enqueued, in the C ABI and in the binding.  CPU only."""
import struct

import pytest
import torch

import bit_microscaled_numerics_amd as nv

FAKE = 0x10000
BF, F, I4, I8 = nv.NVFP4_TYPE_BF16, nv.NVFP4_TYPE_F32, nv.NVFP4_TYPE_I32, nv.NVFP4_TYPE_I64
NULL, SHAPE, ALIGN, ARG = (nv.NVFP4_ERR_NULL, nv.NVFP4_ERR_SHAPE, nv.NVFP4_ERR_ALIGN, nv.NVFP4_ERR_ARG)


@pytest.fixture(scope="module")
def lib():
    return nv.load_library()


def heads(p=FAKE, batch=0, token=0, head=0):
    return struct.pack("4q", p, batch, token, head)


def rope(T=4, Hq=2, Hkv=1, D=16, rot=16, ty=BF, wt=F, it=I8, il=0, norm=1, eps=1e-6, wq=FAKE, wk=FAKE,
         pos=FAKE, inv=FAKE):
    return struct.pack("5q5if4q", T, Hq, Hkv, D, rot, ty, wt, it, il, norm, eps, wq, wk, pos, inv)


Q, K = heads(token=32, head=16), heads(token=16, head=16)
MOVED = heads(p=FAKE + 0x8000, token=32, head=16)


def _rope(lib, q=Q, k=K, qo=Q, ko=K, **kw):
    return lib.nvfp4_qk_norm_rope(rope(**kw), q, k, qo, ko, None)


def _rope_grad(lib, dq=MOVED, dk=K, q=Q, k=K, qo=MOVED, ko=K, dwq=FAKE, dwk=FAKE, ws=FAKE, nb=1 << 22, **kw):
    return lib.nvfp4_qk_norm_rope_grad(rope(**kw), dq, dk, q, k, qo, ko, dwq, dwk, ws, nb, None)


BAD_ROPE = [
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(Hq=-1), SHAPE), (dict(Hkv=1 << 17), SHAPE),
    (dict(D=0, rot=0), SHAPE), (dict(D=15, rot=0), SHAPE), (dict(D=514, rot=2), SHAPE),
    (dict(rot=18), SHAPE), (dict(rot=3), SHAPE), (dict(rot=-2), SHAPE), (dict(ty=I4), ARG), (dict(wt=I8), ARG),
    (dict(it=BF), ARG), (dict(il=2), ARG), (dict(norm=-1), ARG), (dict(norm=0), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(wq=FAKE + 2), ALIGN),
    (dict(pos=0), NULL), (dict(inv=0), NULL), (dict(pos=FAKE + 4), ALIGN), (dict(inv=FAKE + 2), ALIGN),
    (dict(q=None), NULL), (dict(q=heads(p=0)), NULL), (dict(q=heads(p=FAKE + 1, token=32, head=16)), ALIGN),
    (dict(q=heads(token=24, head=16)), SHAPE), (dict(q=heads(token=32, head=8)), SHAPE),
    (dict(q=heads(token=-32, head=16)), SHAPE), (dict(q=heads(token=1 << 39, head=16)), SHAPE),
    (dict(q=heads(token=1 << 62, head=1 << 62)), SHAPE), (dict(ko=None), NULL)]


@pytest.mark.parametrize("kw,status", BAD_ROPE)
def test_rope_refusals(lib, kw, status):
    assert _rope(lib, **kw) == status
    assert lib.nvfp4_last_error()
    assert _rope_grad(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dq=None), NULL), (dict(ws=None), NULL), (dict(ws=FAKE + 8), ALIGN), (dict(nb=10), ARG),
    (dict(dwq=FAKE + 2), ALIGN), (dict(wk=0), ARG), (dict(dk=heads(token=8, head=16)), SHAPE),
    (dict(qo=heads(p=FAKE + 0x8000, token=16, head=64)), ARG)])
def test_rope_grad_refusals(lib, kw, status):
    assert _rope_grad(lib, **kw) == status


def test_rope_in_place_needs_one_layout(lib):
    assert _rope(lib, qo=heads(token=16, head=64)) == ARG


def test_rope_workspace(lib):
    q = lib.nvfp4_qk_norm_rope_grad_workspace_bytes
    assert q(0, 4, 2, 64) == 0 and q(5, 0, 0, 64) == 0
    assert q(-1, 4, 2, 64) == SHAPE and q(4, 4, 2, 63) == SHAPE
    assert 0 < q(8192, 40, 8, 128) <= 1 << 21
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_qk_norm_rope_grad_workspace_bytes(4, 1, 1, 1000)


def attn(batch=2, Tq=4, Tk=6, Hq=4, Hkv=2, D=16, cu_q=0, cu_k=0, it=I4, causal=0, window=0, scale=0.25):
    return struct.pack("8qiiqf4x", batch, Tq, Tk, Hq, Hkv, D, cu_q, cu_k, it, causal, window, scale)


AQ, AK = heads(batch=256, token=64, head=16), heads(batch=192, token=32, head=16)
OQ = heads(p=FAKE + 0x8000, batch=256, token=64, head=16)
GQ = heads(p=FAKE + 0x10000, batch=256, token=64, head=16)
GK, GV = (heads(p=FAKE + n, batch=192, token=32, head=16) for n in (0x18000, 0x20000))


def _attn(lib, q=AQ, k=AK, v=AK, out=OQ, lse=FAKE, ws=FAKE, nb=1 << 40, a=None, **kw):
    return lib.nvfp4_attention(attn(**kw) if a is None else a, q, k, v, out, lse, ws, nb, None)


def _attn_grad(lib, q=AQ, k=AK, v=AK, out=OQ, lse=FAKE, ws=FAKE, nb=1 << 40, dout=AQ, dq=GQ, dk=GK, dv=GV, **kw):
    return lib.nvfp4_attention_grad(attn(**kw), dout, q, k, v, out, lse, dq, dk, dv, ws, nb, None)


BAD_ATTN = [
    (dict(batch=-1), SHAPE), (dict(Tq=-1), SHAPE), (dict(Tk=1 << 31), SHAPE), (dict(Hq=3), SHAPE),
    (dict(Hkv=0), SHAPE), (dict(Hq=0), SHAPE), (dict(Hkv=-2), SHAPE), (dict(Hq=1 << 17, Hkv=1), SHAPE),
    (dict(D=0), SHAPE), (dict(D=12), SHAPE), (dict(D=136), SHAPE), (dict(Tq=1 << 29), SHAPE),
    (dict(batch=1 << 30), SHAPE), (dict(Tk=1 << 30), SHAPE),
    (dict(cu_q=FAKE), ARG), (dict(cu_k=FAKE), ARG), (dict(cu_q=FAKE, cu_k=FAKE, it=BF), ARG),
    (dict(cu_q=FAKE + 2, cu_k=FAKE), ALIGN), (dict(cu_q=FAKE, cu_k=FAKE + 4, it=I8), ALIGN),
    (dict(causal=2), ARG), (dict(window=3), ARG), (dict(window=-1, causal=1), ARG), (dict(scale=0.0), ARG),
    (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
    (dict(scale=2.0 ** -65), ARG), (dict(scale=2.0 ** 65), ARG),
    (dict(q=None), NULL), (dict(k=heads(p=0, batch=192, token=32, head=16)), NULL), (dict(lse=None), NULL),
    (dict(lse=FAKE + 2), ALIGN), (dict(v=heads(p=FAKE + 8, batch=192, token=32, head=16)), ALIGN),
    (dict(q=heads(batch=256, token=68, head=16)), ALIGN), (dict(q=heads(batch=256, token=56, head=16)), SHAPE),
    (dict(k=heads(batch=8, token=32, head=16)), SHAPE), (dict(k=heads(batch=192, token=0, head=16)), SHAPE),
    (dict(k=heads(batch=1 << 30, token=1 << 22, head=16)), SHAPE),
    (dict(q=heads(batch=1 << 34, token=16, head=(1 << 29) + 8)), SHAPE),
    (dict(out=heads(batch=1 << 62, token=64, head=16)), SHAPE)]


@pytest.mark.parametrize("kw,status", BAD_ATTN)
def test_attention_refusals(lib, kw, status):
    assert _attn(lib, **kw) == status
    assert lib.nvfp4_last_error()
    assert _attn_grad(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(ws=None), NULL), (dict(ws=FAKE + 64), ALIGN), (dict(nb=16), ARG), (dict(dout=None), NULL),
    (dict(dq=heads(p=0, batch=256, token=64, head=16)), NULL), (dict(dk=heads(batch=192, token=36, head=16)), ALIGN),
    (dict(dv=heads(batch=192, token=8, head=16)), SHAPE), (dict(dq=AQ), ARG), (dict(dq=OQ), ARG),
    (dict(dk=AK), ARG), (dict(dv=GK), ARG)])
def test_attention_grad_refusals(lib, kw, status):
    assert _attn_grad(lib, **kw) == status


def test_attention_is_not_in_place(lib):
    assert _attn(lib, out=AQ) == ARG


def test_attention_workspace(lib):
    q = lib.nvfp4_attention_workspace_bytes
    assert q(None, 0) == NULL and q(attn(D=9), 0) == SHAPE and q(attn(), 2) == ARG
    assert q(attn(), 1) > 0
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_attention_workspace_bytes(attn(D=9), True)


def test_binding_refuses():
    x = torch.zeros(4, 2, 16, dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        nv.qk_norm_rope(x, x)   # not on a GPU
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        nv.attention(x, x, x)
    for bad in (dict(positions=torch.zeros(4, dtype=torch.int64)), dict(inv_freq=torch.ones(8))):
        with pytest.raises(ValueError):
            nv.qk_norm_rope(x, x, **bad)
    with pytest.raises(ValueError):
        nv.qk_norm_rope(x, x[:3])
    with pytest.raises(ValueError):
        nv.qk_norm_rope(x.half(), x.half())
    with pytest.raises(ValueError):
        nv.attention(x, x, x[:3])
    with pytest.raises(ValueError):
        nv.attention(x, x[..., :8], x[..., :8])
    with pytest.raises(ValueError):
        nv.attention(x, x, x, cu_k=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        nv.attention(x[None], x, x)
