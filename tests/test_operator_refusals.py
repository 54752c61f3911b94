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


def test_fp4_products_reject(lib):
    nan, inf = float("nan"), float("inf")
    gemm = dict(x=F, xs=F, rows=2048, K=2880, b=F, s=F, E=32, N=5760, k=4, off=F, sp=F, tl=F, nt=F,
                mt=32 + 33 + 1, tm=256, out=F)
    head, tail = "x xs rows K b s E N k".split(), "off sp tl nt mt tm out".split()
    plain = _caller(lib.gq_mxfp4_grouped_gemm_fp4, head + ["ps"] + tail, dict(gemm, ps=NULL))
    unit = _caller(lib.gq_mxfp4_grouped_gemm_fp4_swiglu, head + ["al", "li"] + tail,
                   dict(gemm, al=1.702, li=7.0))
    for call in (plain, unit):
        for bad in (dict(x=NULL), dict(xs=NULL), dict(b=NULL), dict(s=NULL), dict(off=NULL),
                    dict(sp=NULL), dict(tl=NULL), dict(nt=NULL), dict(out=NULL), dict(rows=-1),
                    dict(K=0), dict(K=2870), dict(N=0), dict(N=5750), dict(E=0), dict(k=0),
                    dict(mt=64), dict(x=F8), dict(b=F8), dict(out=F8), dict(off=F2), dict(nt=F2)):
            assert call(**bad) == INVALID, bad
        assert call(tm=128) == NOT_SUPPORTED
        assert call(rows=1 << 21, mt=1 << 24) == NOT_SUPPORTED     # 32-bit row offsets
        assert call(N=1 << 21) == NOT_SUPPORTED                    # 32-bit offsets in an expert
        assert call(rows=0) == 0
    for bad in (dict(al=nan), dict(al=inf), dict(li=-1.0), dict(li=nan), dict(li=inf)):
        assert unit(**bad) == INVALID, bad
    assert plain(ps=F2) == INVALID
    gemv = dict(x=F, xs=F, rows=1, K=2880, b=F, s=F, E=32, N=5760, ids=F, k=4, out=F)
    head = "x xs rows K b s E N ids k".split()
    plain = _caller(lib.gq_mxfp4_grouped_gemv_fp4, head + ["ps", "out"], dict(gemv, ps=NULL))
    unit = _caller(lib.gq_mxfp4_grouped_gemv_fp4_swiglu, head + ["al", "li", "out"],
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


def _layer(**kw):
    """A layer struct of fake pointers (topk 4 of 32 MXFP4 experts)."""
    a = dict(format=1, num_experts=32, topk=4, hidden=2880, inner=2880, renormalize=1, alpha=1.702,
             limit=7.0, router_weight=0x1000, router_bias=None, gate_up_codes=0x1000,
             gate_up_scales=0x1000, gate_up_bias=None, down_codes=0x1000, down_scales=0x1000,
             down_bias=None)
    a.update(kw)
    return gq._LayerStruct(**a)


def test_moe_decode_rejects(lib):
    def call(x=F, rows=1, xs=2880, ws=F, nbytes=1 << 30, y=F, **kw):
        return lib.gq_moe_decode(ctypes.byref(_layer(**kw)), x, rows, xs, ws, nbytes, y, None)

    nan, inf = float("nan"), float("inf")
    for bad in (dict(x=NULL), dict(y=NULL), dict(ws=NULL), dict(rows=-1), dict(xs=2879),
                dict(xs=2884), dict(x=F8), dict(ws=F8), dict(y=F1), dict(nbytes=100),
                dict(format=2), dict(num_experts=0), dict(topk=0), dict(topk=33), dict(hidden=0),
                dict(hidden=2896, xs=2896), dict(inner=2896), dict(inner=-32), dict(alpha=nan),
                dict(alpha=inf), dict(limit=-1.0), dict(limit=inf), dict(limit=nan),
                dict(router_weight=None), dict(gate_up_codes=None), dict(gate_up_scales=None),
                dict(down_codes=None), dict(down_scales=None), dict(router_weight=0x1008),
                dict(gate_up_codes=0x1004), dict(down_codes=0x1008), dict(router_bias=0x1001),
                dict(gate_up_bias=0x1001), dict(down_bias=0x1001)):
        assert call(**bad) == INVALID, bad
    assert call(format=0, inner=2912) == INVALID              # NF4: multiples of 64
    assert call(format=0, gate_up_scales=0x1002) == INVALID
    for bad in (dict(rows=9), dict(rows=8, topk=9), dict(num_experts=513), dict(inner=4128),
                dict(hidden=8224, xs=8224), dict(xs=1 << 31)):
        assert call(**bad) == NOT_SUPPORTED, bad
    assert call(rows=0, x=NULL, y=NULL, ws=NULL) == 0
    assert lib.gq_moe_decode(None, F, 1, 2880, F, 1 << 30, F, None) == INVALID


def test_moe_decode_workspace_sizes(lib):
    size = lambda rows, **kw: lib.gq_moe_decode_workspace(ctypes.byref(_layer(**kw)), rows)  # noqa: E731
    assert size(0) == 0
    assert size(1) >= 4 * (32 + 2 * 4 + 4 * 2880)
    assert size(8) > size(1)
    for bad in (dict(rows=-1), dict(rows=9), dict(rows=8, topk=9), dict(rows=1, hidden=100),
                dict(rows=1, num_experts=600)):
        assert size(**bad) == -1, bad
    assert lib.gq_moe_decode_workspace(None, 1) == -1
    # a workspace one byte short is refused before anything is enqueued
    need = size(2)
    assert lib.gq_moe_decode(ctypes.byref(_layer()), F, 2, 2880, F, need - 1, F, None) == INVALID


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


def test_short_calls_leave_what_is_not_ordinary(lib):
    """The short calls return None, and touch nothing, for what is not a plain
    device tensor; the Python code then refuses it."""
    calls = gq._calls
    assert calls is not None and calls.torch_version == torch.__version__
    x = torch.zeros(4, 64)
    i = torch.zeros(4, 2, dtype=torch.int32)
    assert calls.quantize(x, False) is None
    assert calls.quantize(None, True) is None
    assert calls.moe_topk(x, 2, True) is None
    assert calls.moe_topk("x", 2, True) is None
    assert calls.moe_topk_backward(torch.zeros(4, 2), x, i, True) is None
    assert calls.route_sort(i, 4, 256) is None
    assert calls.fp4_gemv(x, x, x, x, i, None, False, 0.0, 0.0) is None
    assert calls.fp4_gemm(x, x, x, x, (), None, True, 1.0, 1.0) is None
    assert calls.moe_decode(0, 0, 16, x) is None
    for f in (calls.quantize, calls.moe_topk, calls.route_sort, calls.fp4_gemm, calls.bind):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(KeyError):
        calls.bind({}, None, None)
    gq._load_calls(lib)                                   # bound again as it was


def test_launches_that_the_runtime_does_not_take(lib):
    """A launch takes fewer than 2^32 threads along a dimension: the product
    refuses tile lists of 2^24 workgroups or more."""
    head, tail = "x xs rows K b s E N k".split(), "off sp tl nt mt tm out".split()
    base = dict(x=F, xs=F, rows=1 << 26, K=32, b=F, s=F, E=32, N=32, k=16, off=F, sp=F, tl=F, nt=F,
                mt=(1 << 22) + 64, tm=256, out=F)          # 2^30 pairs, four workgroups a tile
    plain = _caller(lib.gq_mxfp4_grouped_gemm_fp4, head + ["ps"] + tail, dict(base, ps=NULL))
    unit = _caller(lib.gq_mxfp4_grouped_gemm_fp4_swiglu, head + ["al", "li"] + tail,
                   dict(base, al=1.702, li=7.0))
    for call in (plain, unit):
        assert call() == NOT_SUPPORTED
        assert call(rows=2048, k=4, mt=1 << 22) == NOT_SUPPORTED
        assert call(rows=2048, k=4, N=1025, mt=1 << 21) == INVALID       # N % 32
        assert call(rows=2048, k=4, N=1056, mt=1 << 21) == NOT_SUPPORTED
    for rows, E in (((1 << 33) + 1, 1), ((1 << 33) + 1, 300)):
        f = _caller(lib.gq_moe_topk, "z dt rows E zs k renorm ids w".split(),
                    dict(z=F, dt=0, rows=rows, E=E, zs=E, k=1, renorm=1, ids=F, w=F))
        b = _caller(lib.gq_moe_topk_backward, "dw z dt rows E zs ids k renorm dz".split(),
                    dict(dw=F, z=F, dt=1, rows=rows, E=E, zs=E, ids=F, k=1, renorm=0, dz=F))
        assert f() == NOT_SUPPORTED and b() == NOT_SUPPORTED


def test_sizes_past_32_bits_are_not_cut_short(lib):
    """The library takes sizes in 32 bits; a larger one is refused, not passed
    on as its low half."""
    layer = gq.MoeLayer(_layer(), (), torch.device("cuda", 0))
    assert gq.gq_moe_decode_workspace(layer, 1) > 0
    for rows in ((1 << 32) + 1, 1 << 31, 1 << 40, 1 - (1 << 32)):
        assert gq.gq_moe_decode_workspace(layer, rows) == -1
    for bad in (((1 << 32) + 4, 2, 8), (4, (1 << 32) + 2, 8), (4, 2, (1 << 32) + 8),
                (4, 2, 8, (1 << 32) + 256)):
        with pytest.raises(gq.GQError):
            gq.gq_route_max_tiles(*bad)
    assert gq.gq_route_max_tiles(-1, 2, 8) == -1
    gq._ints("sizes", 0, -1, (1 << 31) - 1, -(1 << 31))
    for n in (1 << 31, -(1 << 31) - 1, (1 << 32) + 1):
        with pytest.raises(gq.GQError, match="not supported"):
            gq._ints("sizes", 1, n)


def test_a_layer_keeps_the_memory_that_it_names():
    """A tensor given other memory leaves the layer's addresses valid."""
    weight = torch.nn.Parameter(torch.arange(8.0))
    was = weight.data_ptr()
    layer = gq.MoeLayer(_layer(router_weight=was), (weight, None), torch.device("cpu"))
    weight.data = torch.zeros(8)
    assert weight.data_ptr() != was
    assert [t.data_ptr() for t in layer._tensors if t is not None] == [was]
    assert torch.equal(layer._tensors[0], torch.arange(8.0))
    assert not layer._tensors[0].requires_grad
