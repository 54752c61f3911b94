"""What the quantiser, the router and the layer entry points refuse, on the
host: malformed arguments to the C ABI (nothing is enqueued, no GPU is
needed) and to the Python binding."""

import ctypes

import pytest
import torch

import bit_grouped_moe_amd as gq

INVALID, NOT_SUPPORTED = 1, 801
F = ctypes.c_void_p(0x1000)          # a fake, aligned, never-dereferenced pointer
F1 = ctypes.c_void_p(0x1001)
F2 = ctypes.c_void_p(0x1002)
F8 = ctypes.c_void_p(0x1008)
NULL = None


@pytest.fixture(scope="module")
def lib():
    return gq.load_library()


def _caller(fn, names, ok):
    def call(**kw):
        assert set(kw) <= set(names)
        return fn(*[{**ok, **kw}[n] for n in names], None)
    return call


def test_quantize_rejects(lib):
    call = _caller(lib.gq_mxfp4_quantize, "x dt rows K xs b s v".split(),
                   dict(x=F, dt=1, rows=4, K=64, xs=64, b=F, s=F, v=NULL))
    for bad in (dict(x=NULL), dict(b=NULL), dict(s=NULL), dict(dt=3), dict(dt=-1), dict(rows=-1),
                dict(K=0), dict(K=-32), dict(K=48), dict(xs=63), dict(xs=0), dict(xs=-64),
                dict(x=F1), dict(x=F2, dt=0), dict(b=F8), dict(v=F8)):
        assert call(**bad) == INVALID, bad
    assert call(xs=1 << 62) == NOT_SUPPORTED
    assert call(rows=1 << 40, K=1 << 20, xs=1 << 20) == NOT_SUPPORTED
    assert call(rows=0, x=NULL, b=NULL, s=NULL) == 0


def test_moe_topk_rejects(lib):
    call = _caller(lib.gq_moe_topk, "z dt rows E zs k renorm ids w".split(),
                   dict(z=F, dt=0, rows=4, E=128, zs=128, k=8, renorm=1, ids=F, w=F))
    for bad in (dict(z=NULL), dict(ids=NULL), dict(w=NULL), dict(dt=7), dict(rows=-1), dict(E=0),
                dict(k=0), dict(k=129), dict(zs=127), dict(z=F2), dict(z=F1, dt=1), dict(ids=F2),
                dict(w=F2)):
        assert call(**bad) == INVALID, bad
    assert call(E=1025, zs=1025) == NOT_SUPPORTED
    assert call(k=65) == NOT_SUPPORTED
    assert call(rows=1 << 40) == NOT_SUPPORTED
    assert call(rows=0, z=NULL, ids=NULL, w=NULL) == 0


def test_moe_topk_backward_rejects(lib):
    call = _caller(lib.gq_moe_topk_backward, "dw z dt rows E zs ids k renorm dz".split(),
                   dict(dw=F, z=F, dt=1, rows=4, E=32, zs=32, ids=F, k=4, renorm=0, dz=F))
    for bad in (dict(dw=NULL), dict(z=NULL), dict(ids=NULL), dict(dz=NULL), dict(dt=3),
                dict(rows=-1), dict(E=0), dict(k=0), dict(zs=31), dict(dw=F2),
                dict(z=F1), dict(ids=F2), dict(dz=F1), dict(dz=F2, dt=0, z=F)):
        assert call(**bad) == INVALID, bad
    assert call(E=2000, zs=2000) == NOT_SUPPORTED
    assert call(k=65) == NOT_SUPPORTED
    assert call(rows=0) == 0


def test_binding_refuses_host_tensors_and_wrong_types(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        gq.gq_mxfp4_quantize(x)
    with pytest.raises(ValueError, match="device tensor"):
        gq.gq_moe_topk(x, 2)
    with pytest.raises(ValueError, match="device tensor"):
        gq.gq_moe_topk_backward(torch.zeros(4, 2), x, torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        gq.gq_mxfp4_quantize([1.0])


def test_row_layouts():
    """Row stride of [..., width] tensors; layouts without one are refused."""
    x = torch.zeros(6, 4, 32)
    assert gq._rows(x, "x") == (24, 32, 32)
    assert gq._rows(x[:, 0], "x") == (6, 32, 128)
    assert gq._rows(x[0, 0], "x") == (1, 32, 32)
    assert gq._rows(torch.zeros(32, 1).t(), "x") == (1, 32, 32)
    assert gq._rows(torch.zeros(0, 32), "x") == (0, 32, 32)
    for bad in (x[:, :2], x[..., ::2], x.transpose(0, 2)):
        with pytest.raises(ValueError):
            gq._rows(bad, "x")
