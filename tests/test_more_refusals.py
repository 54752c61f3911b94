"""What the norm, the 8-bit quantiser, the routing with groups and the 8-bit
products refuse, on the host: malformed arguments to the C ABI (nothing is
enqueued, no GPU is needed) and to the Python binding."""

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
    call = _caller(lib.gq_mxfp8_quantize, "x dt rows K xs c s v".split(),
                   dict(x=F, dt=1, rows=4, K=64, xs=64, c=F, s=F, v=NULL))
    for bad in (dict(x=NULL), dict(c=NULL), dict(s=NULL), dict(dt=3), dict(dt=-1), dict(rows=-1),
                dict(K=0), dict(K=-32), dict(K=48), dict(xs=63), dict(xs=0), dict(xs=-64),
                dict(x=F1), dict(x=F2, dt=0), dict(c=F8), dict(v=F8)):
        assert call(**bad) == INVALID, bad
    assert call(xs=1 << 62) == NOT_SUPPORTED
    assert call(rows=0, x=NULL, c=NULL, s=NULL) == 0


def test_norm_rejects(lib):
    call = _caller(lib.gq_rms_norm, "x xs r rs dt rows H w wdt eps sum y c s v".split(),
                   dict(x=F, xs=64, r=F, rs=64, dt=1, rows=4, H=64, w=F, wdt=1, eps=1e-6, sum=F,
                        y=F, c=F, s=F, v=F))
    nan, inf = float("nan"), float("inf")
    for bad in (dict(x=NULL), dict(w=NULL), dict(dt=3), dict(wdt=2), dict(wdt=3), dict(dt=0, x=F),
                dict(rows=-1), dict(H=0), dict(H=-64), dict(xs=63), dict(rs=63), dict(rs=0),
                dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(r=NULL), dict(c=NULL),
                dict(s=NULL), dict(c=NULL, s=NULL), dict(H=63), dict(x=F1), dict(r=F1), dict(w=F1),
                dict(sum=F1), dict(y=F1), dict(c=F8), dict(v=F8),
                dict(w=F2, wdt=0), dict(sum=NULL, y=NULL, c=NULL, s=NULL, v=NULL)):
        assert call(**bad) == INVALID, bad
    assert call(H=32800, xs=32800, rs=32800) == NOT_SUPPORTED
    assert call(xs=1 << 62) == NOT_SUPPORTED
    assert call(rs=1 << 62) == NOT_SUPPORTED
    assert call(rows=1 << 50, H=32768, xs=32768, rs=32768) == NOT_SUPPORTED
    assert call(rows=0, x=NULL, w=NULL, y=NULL) == 0


def test_outputs_in_place_of_strided_inputs(lib):
    """In place only where rows do not lie at another stride; the same for both
    of a norm's outputs and for the gradient."""
    G, D = ctypes.c_void_p(0x200000), ctypes.c_void_p(0x300000)
    call = _caller(lib.gq_rms_norm, "x xs r rs dt rows H w wdt eps sum y c s v".split(),
                   dict(x=F, xs=72, r=G, rs=80, dt=1, rows=4, H=64, w=F, wdt=1, eps=1e-6,
                        sum=NULL, y=NULL, c=NULL, s=NULL, v=NULL))
    for bad in (dict(y=F), dict(sum=F), dict(y=G), dict(sum=G), dict(sum=D, y=D),
                dict(sum=F, y=F, xs=64), dict(y=F, rows=2)):
        assert call(**bad) == INVALID, bad
    call = _caller(lib.gq_rms_norm_backward,
                   "dy dys h hs dh dhs dt rows H w wdt eps dx dw ws wn".split(),
                   dict(dy=F, dys=72, h=G, hs=72, dh=D, dhs=72, dt=2, rows=4, H=64, w=F, wdt=2,
                        eps=1e-6, dx=F, dw=NULL, ws=NULL, wn=0))
    for bad in (dict(dx=F), dict(dx=G), dict(dx=D)):
        assert call(**bad) == INVALID, bad


def test_norm_backward_rejects(lib):
    call = _caller(lib.gq_rms_norm_backward,
                   "dy dys h hs dh dhs dt rows H w wdt eps dx dw ws wn".split(),
                   dict(dy=F, dys=64, h=F, hs=64, dh=F, dhs=64, dt=2, rows=4, H=64, w=F, wdt=2,
                        eps=1e-6, dx=F, dw=F, ws=F, wn=1 << 30))
    for bad in (dict(dy=NULL), dict(h=NULL), dict(w=NULL), dict(dx=NULL), dict(ws=NULL),
                dict(wn=64 * 4 - 1), dict(ws=F8), dict(dt=3), dict(wdt=1), dict(rows=-1),
                dict(H=0), dict(dys=63), dict(hs=63), dict(dhs=63), dict(eps=-1e-6), dict(dy=F1),
                dict(h=F1), dict(dh=F1), dict(w=F1), dict(dx=F1), dict(dw=F1),
                dict(dw=F2, wdt=0)):
        assert call(**bad) == INVALID, bad
    assert call(H=32769, dys=32769, hs=32769, dhs=32769) == NOT_SUPPORTED
    assert call(hs=1 << 62) == NOT_SUPPORTED
    assert call(dhs=1 << 62) == NOT_SUPPORTED
    assert call(rows=0, dw=NULL) == 0
    assert lib.gq_rms_norm_backward_workspace(-1, 64) == -1
    assert lib.gq_rms_norm_backward_workspace(4, 0) == -1
    assert lib.gq_rms_norm_backward_workspace(4, 32769) == -1
    assert lib.gq_rms_norm_backward_workspace(0, 64) == 0
    assert gq.gq_rms_norm_backward_workspace(1 << 70, 64) == -1
    assert gq.gq_rms_norm_backward_workspace(4, 1 << 40) == -1


def test_fp8_products_reject(lib):
    nan, inf = float("nan"), float("inf")
    gemm = dict(x=F, xs=F, rows=2048, K=2880, b=F, s=F, E=32, N=5760, k=4, off=F, sp=F, tl=F, nt=F,
                mt=32 + 33 + 1, tm=256, out=F)
    head, tail = "x xs rows K b s E N k".split(), "off sp tl nt mt tm out".split()
    plain = _caller(lib.gq_mxfp4_grouped_gemm_fp8, head + ["ps"] + tail, dict(gemm, ps=NULL))
    unit = _caller(lib.gq_mxfp4_grouped_gemm_fp8_swiglu, head + ["al", "li"] + tail,
                   dict(gemm, al=1.702, li=7.0))
    for call in (plain, unit):
        for bad in (dict(x=NULL), dict(xs=NULL), dict(b=NULL), dict(s=NULL), dict(off=NULL),
                    dict(sp=NULL), dict(tl=NULL), dict(nt=NULL), dict(out=NULL), dict(rows=-1),
                    dict(K=0), dict(K=2870), dict(N=0), dict(N=5750), dict(E=0), dict(k=0),
                    dict(mt=64), dict(x=F8), dict(b=F8), dict(out=F8), dict(off=F2), dict(nt=F2)):
            assert call(**bad) == INVALID, bad
        assert call(tm=128) == NOT_SUPPORTED
        assert call(rows=1 << 20, mt=1 << 24) == NOT_SUPPORTED     # 32-bit row offsets
        assert call(N=1 << 21) == NOT_SUPPORTED                    # 32-bit offsets in an expert
        assert call(rows=0) == 0
    for bad in (dict(al=nan), dict(al=inf), dict(li=-1.0), dict(li=nan), dict(li=inf)):
        assert unit(**bad) == INVALID, bad
    assert plain(ps=F2) == INVALID
    gemv = dict(x=F, xs=F, rows=1, K=2880, b=F, s=F, E=32, N=5760, ids=F, k=4, out=F)
    head = "x xs rows K b s E N ids k".split()
    plain = _caller(lib.gq_mxfp4_grouped_gemv_fp8, head + ["ps", "out"], dict(gemv, ps=NULL))
    unit = _caller(lib.gq_mxfp4_grouped_gemv_fp8_swiglu, head + ["al", "li", "out"],
                   dict(gemv, al=1.702, li=7.0))
    for call in (plain, unit):
        for bad in (dict(x=NULL), dict(xs=NULL), dict(b=NULL), dict(s=NULL), dict(ids=NULL),
                    dict(out=NULL), dict(rows=0), dict(K=0), dict(K=2870), dict(N=0), dict(E=0),
                    dict(k=0), dict(x=F8), dict(b=F8), dict(ids=F2)):
            assert call(**bad) == INVALID, bad
        assert call(rows=65) == NOT_SUPPORTED
        assert call(K=8224) == NOT_SUPPORTED
    assert unit(N=5761) == INVALID
    assert unit(al=nan) == INVALID and unit(li=-1.0) == INVALID


def test_moe_route_rejects(lib):
    call = _caller(lib.gq_moe_route, "z dt rows E zs b k sc G kG top renorm f ids w".split(),
                   dict(z=F, dt=0, rows=4, E=256, zs=256, b=F, k=8, sc=1, G=8, kG=4, top=2,
                        renorm=1, f=2.5, ids=F, w=F))
    nan, inf = float("nan"), float("inf")
    for bad in (dict(z=NULL), dict(ids=NULL), dict(w=NULL), dict(dt=7), dict(rows=-1), dict(E=0),
                dict(k=0), dict(k=129), dict(zs=255), dict(z=F2), dict(z=F1, dt=1), dict(ids=F2),
                dict(w=F2), dict(b=F2), dict(sc=2), dict(sc=-1), dict(G=0), dict(G=-8), dict(G=7),
                dict(kG=0), dict(kG=9), dict(top=0), dict(top=3), dict(f=nan), dict(f=inf),
                dict(f=-inf)):
        assert call(**bad) == INVALID, bad
    assert call(E=1032, zs=1032) == NOT_SUPPORTED
    assert call(k=65) == NOT_SUPPORTED
    assert call(G=128, kG=64) == NOT_SUPPORTED
    assert call(rows=1 << 40) == NOT_SUPPORTED
    assert call(rows=0, z=NULL, ids=NULL, w=NULL) == 0


def test_moe_route_backward_rejects(lib):
    call = _caller(lib.gq_moe_route_backward, "dw z dt rows E zs ids k sc renorm f dz".split(),
                   dict(dw=F, z=F, dt=1, rows=4, E=32, zs=32, ids=F, k=4, sc=1, renorm=0, f=1.0,
                        dz=F))
    for bad in (dict(dw=NULL), dict(z=NULL), dict(ids=NULL), dict(dz=NULL), dict(dt=3),
                dict(rows=-1), dict(E=0), dict(k=0), dict(zs=31), dict(dw=F2), dict(sc=2),
                dict(sc=-1), dict(f=float("nan")), dict(f=float("inf")), dict(z=F1), dict(ids=F2),
                dict(dz=F1), dict(dz=F2, dt=0, z=F)):
        assert call(**bad) == INVALID, bad
    assert call(E=2000, zs=2000) == NOT_SUPPORTED
    assert call(k=65) == NOT_SUPPORTED
    assert call(rows=0) == 0


def test_binding_takes_device_tensors_only():
    x, w = torch.zeros(2, 64), torch.ones(64)
    for call in (lambda: gq.gq_mxfp8_quantize(x), lambda: gq.gq_rms_norm(x, w),
                 lambda: gq.gq_rms_norm_backward(x, x, w), lambda: gq.gq_moe_route(x, 2),
                 lambda: gq.gq_moe_route_backward(x, x, x)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gq.gq_mxfp8_quantize(None), lambda: gq.gq_rms_norm([1.0], w),
                 lambda: gq.gq_rms_norm_backward(x, None, w)):
        with pytest.raises(TypeError):
            call()
