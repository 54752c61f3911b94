"""The binding's two ways to the library, short calls and Python code, give
the same outputs and refuse the same arguments with the same errors."""

import numpy as np
import pytest
import torch

import bit_grouped_moe_amd as gq
import workloads as wl
from tests.gpu_common import device, packed_mx_bank, say, to_dev, to_dev_bf16

pytestmark = pytest.mark.gpu


def _both(monkeypatch, f):
    """f() with the short calls and without: outputs, or the error of each."""
    def once():
        try:
            return f()
        except Exception as e:                            # compared, not swallowed
            return type(e), str(e)
    assert gq._calls is not None, "the short calls are not built"
    fast = once()
    with monkeypatch.context() as m:
        m.setattr(gq, "_calls", None)
        slow = once()
    torch.cuda.synchronize()
    return fast, slow


def _same(a, b):
    if isinstance(a, torch.Tensor):
        assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)
    elif isinstance(a, tuple):
        assert len(a) == len(b) and type(a) is type(b)
        for x, y in zip(a, b):
            _same(x, y)
    else:
        assert a == b


class Operands:
    def __init__(self):
        dev = device()
        g = np.random.default_rng(8)
        self.x = to_dev_bf16(wl.draw_bf16(g, (6, 96)), dev)
        self.bank = tuple(to_dev(t, dev) for t in packed_mx_bank(g, 4, 64, 96))
        self.down = tuple(to_dev(t, dev) for t in packed_mx_bank(g, 4, 96, 32))
        self.ids = to_dev(wl.route_uniform(g, 6, 4, 2), dev)
        self.z = torch.from_numpy(g.standard_normal((6, 4)).astype(np.float32)).to(dev)
        self.w = torch.rand(12, device=dev)
        self.router = to_dev_bf16(wl.draw_bf16(g, (4, 96)), dev)


def test_same_outputs(monkeypatch):
    o = Operands()
    say("calls: outputs")
    q = gq.gq_mxfp4_quantize(o.x)
    route = gq.gq_route_sort(o.ids, 4)
    layer = gq.gq_moe_layer(o.router, o.bank, o.down, 2)
    gq.gq_moe_decode(layer, o.x)                          # the workspace size is known from here on
    wide = torch.zeros(6, 128, dtype=torch.float16, device=o.x.device)
    ids, _ = gq.gq_moe_topk(o.z, 2)
    for f in (lambda: gq.gq_mxfp4_quantize(o.x), lambda: gq.gq_mxfp4_quantize(o.x, values=True),
              lambda: gq.gq_mxfp4_quantize(wide[:, 3:99]), lambda: gq.gq_mxfp4_quantize(o.x[0]),
              lambda: gq.gq_mxfp4_quantize(o.x.float().reshape(2, 3, 96), values=True),
              lambda: gq.gq_mxfp4_quantize(o.x[:0]),
              lambda: gq.gq_moe_topk(o.z, 2), lambda: gq.gq_moe_topk(o.z[:, 1:3], 1, False),
              lambda: gq.gq_moe_topk(o.z[:1], 4), lambda: gq.gq_moe_topk(o.z[:0], 4),
              lambda: gq.gq_moe_topk_backward(o.w.reshape(6, 2), o.z, ids),
              lambda: gq.gq_moe_topk_backward(o.w.reshape(6, 2), o.z.half(), ids, False),
              lambda: gq.gq_route_sort(o.ids, 4), lambda: gq.gq_route_sort(o.ids, 3, 64),
              lambda: gq.gq_route_sort(o.ids[:0], 4),
              lambda: gq.gq_mxfp4_grouped_gemv_fp4(q, *o.bank, o.ids),
              lambda: gq.gq_mxfp4_grouped_gemv_fp4(q, *o.bank, o.ids, pair_scale=o.w),
              lambda: gq.gq_mxfp4_grouped_gemv_fp4_swiglu(q, *o.bank, o.ids, limit=2.0),
              lambda: gq.gq_mxfp4_grouped_gemm_fp4(q, *o.bank, route),
              lambda: gq.gq_mxfp4_grouped_gemm_fp4(q, *o.bank, route, pair_scale=o.w),
              lambda: gq.gq_mxfp4_grouped_gemm_fp4_swiglu(q, *o.bank, route, alpha=1, limit=3),
              lambda: gq.gq_moe_decode(layer, o.x), lambda: gq.gq_moe_decode(layer, o.x[2:3])):
        fast, slow = _both(monkeypatch, f)
        assert not (isinstance(fast, tuple) and isinstance(fast[0], type)), fast
        _same(fast, slow)


def test_same_refusals(monkeypatch):
    o = Operands()
    say("calls: refusals")
    q = gq.gq_mxfp4_quantize(o.x)
    route = gq.gq_route_sort(o.ids, 4)
    layer = gq.gq_moe_layer(o.router, o.bank, o.down, 2)
    gq.gq_moe_decode(layer, o.x)
    cpu = o.x.cpu()
    nan = float("nan")
    for f in (lambda: gq.gq_mxfp4_quantize(cpu), lambda: gq.gq_mxfp4_quantize(None),
              lambda: gq.gq_mxfp4_quantize(o.x[:, :40]), lambda: gq.gq_mxfp4_quantize(o.x[:, ::2]),
              lambda: gq.gq_mxfp4_quantize(o.ids), lambda: gq.gq_mxfp4_quantize(o.x.t()),
              lambda: gq.gq_mxfp4_quantize(o.x[:1].expand(6, 96)),
              lambda: gq.gq_moe_topk(o.z, 0), lambda: gq.gq_moe_topk(o.z, 5),
              lambda: gq.gq_moe_topk(o.z[0], 2), lambda: gq.gq_moe_topk(o.z.double(), 2),
              lambda: gq.gq_moe_topk(o.z, 1 << 70),
              lambda: gq.gq_moe_topk_backward(o.w, o.z, o.ids),
              lambda: gq.gq_moe_topk_backward(o.w.reshape(6, 2), o.z, o.ids.long()),
              lambda: gq.gq_route_sort(o.ids, 0), lambda: gq.gq_route_sort(o.ids, 2000),
              lambda: gq.gq_route_sort(o.ids.long(), 4),
              lambda: gq.gq_mxfp4_grouped_gemv_fp4(q, *o.bank, o.ids[:4]),
              lambda: gq.gq_mxfp4_grouped_gemv_fp4(q, *o.bank, o.ids, pair_scale=o.w[:3]),
              lambda: gq.gq_mxfp4_grouped_gemv_fp4(q, o.bank[0], o.bank[0], o.ids),
              lambda: gq.gq_mxfp4_grouped_gemv_fp4_swiglu(q, *o.bank, o.ids, alpha=nan),
              lambda: gq.gq_mxfp4_grouped_gemm_fp4(q, *o.down, route),
              lambda: gq.gq_mxfp4_grouped_gemm_fp4(q, *o.bank, route._replace(tile_m=128)),
              lambda: gq.gq_mxfp4_grouped_gemm_fp4(q, *o.bank, route._replace(max_tiles=1)),
              lambda: gq.gq_mxfp4_grouped_gemm_fp4(
                  q, *o.bank, route._replace(tiles=route.tiles.long())),
              lambda: gq.gq_mxfp4_grouped_gemm_fp4(q, *o.bank, route._replace(topk=3)),
              lambda: gq.gq_mxfp4_grouped_gemm_fp4(q, *o.bank, route._replace(max_tiles=1000)),
              lambda: gq.gq_mxfp4_grouped_gemm_fp4(
                  q, *o.bank, route._replace(expert_offsets=route.expert_offsets[:4])),
              lambda: gq.gq_mxfp4_grouped_gemm_fp4_swiglu(q, *o.bank, route, limit=-1.0),
              lambda: gq.gq_moe_decode(layer, cpu), lambda: gq.gq_moe_decode(layer, o.x.float()),
              lambda: gq.gq_moe_decode(layer, o.x[:, :64]), lambda: gq.gq_moe_decode(layer, [1]),
              lambda: gq.gq_moe_decode(layer, torch.cat([o.x, o.x]))):
        fast, slow = _both(monkeypatch, f)
        assert isinstance(fast, tuple) and isinstance(fast[0], type), fast
        assert fast == slow


def test_a_stream_of_its_own(monkeypatch):
    """The short calls use torch's current stream."""
    o = Operands()
    say("calls: side stream")
    x = torch.randn(4096, 2880, device=o.x.device).to(torch.bfloat16)
    ref = gq.gq_mxfp4_quantize(x, values=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = x * 2                                          # on s, before the call
        got = gq.gq_mxfp4_quantize(y, values=True)
    s.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[2], ref[2] * 2)


def test_outputs_are_ordinary_tensors(tmp_path):
    """The outputs of a call share one allocation: they do not overlap, and
    each can be written, differentiated, saved, copied and viewed by itself."""
    import copy
    o = Operands()
    say("calls: outputs as tensors")
    ids, w = gq.gq_moe_topk(o.z, 2)
    blocks, scales = gq.gq_mxfp4_quantize(o.x)
    route = gq.gq_route_sort(o.ids, 4)
    for group in ((ids, w), (blocks, scales), route[:4]):
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in group)
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
        assert all(t.is_contiguous() and t.data_ptr() % 16 == 0 for t in group)
        assert all(not t.requires_grad and t.is_leaf for t in group)
    keep, was = ids.clone(), w.clone()
    w.mul_(3)
    assert torch.equal(ids, keep) and torch.equal(w, was * 3)
    ids.fill_(7)
    assert torch.equal(w, was * 3)
    w.copy_(was)
    w.requires_grad_()
    (w.view(-1) * torch.arange(12.0, device=w.device)).sum().backward()
    assert torch.equal(w.grad.flatten().cpu(), torch.arange(12.0))
    s = scales.clone()
    torch.save(scales, tmp_path / "scales.pt")
    assert torch.equal(torch.load(tmp_path / "scales.pt", weights_only=True), s)
    assert torch.equal(copy.deepcopy(scales), s)
    blocks.zero_()
    assert torch.equal(scales, s)
    with torch.inference_mode():
        ids, w = gq.gq_moe_topk(o.z, 2)
        assert w.is_inference() and torch.equal(w, was)
    assert torch.equal(torch.stack([s, s])[1], s) and scales.untyped_storage().nbytes() > 0


def test_function_transforms_raise_alike(monkeypatch):
    """Tensors without storage (torch.func.vmap) and outputs without storage
    (torch.func.grad): the same error from both ways."""
    o = Operands()
    say("calls: function transforms")
    layer = gq.gq_moe_layer(o.router, o.bank, o.down, 2)
    gq.gq_moe_decode(layer, o.x)
    xb, xs = gq.gq_mxfp4_quantize(o.x)
    route = gq.gq_route_sort(o.ids, 4)
    w = o.w.reshape(6, 2)
    for f, args in ((lambda x: gq.gq_mxfp4_quantize(x, values=True), (o.x,)),
                    (lambda z: gq.gq_moe_topk(z, 2), (o.z,)),
                    (lambda w, z, i: gq.gq_moe_topk_backward(w, z, i), (w, o.z, o.ids)),
                    (lambda i: gq.gq_route_sort(i, 4), (o.ids,)),
                    (lambda x: gq.gq_moe_decode(layer, x), (o.x,)),
                    (lambda b, s, i: gq.gq_mxfp4_grouped_gemv_fp4((b, s), *o.bank, i),
                     (xb, xs, o.ids)),
                    (lambda b, s: gq.gq_mxfp4_grouped_gemm_fp4((b, s), *o.bank, route), (xb, xs))):
        batched = [torch.stack([t, t]) for t in args]

        def in_grad(s):
            f(*args)
            return s * 2
        fast, slow = _both(monkeypatch, lambda: torch.func.vmap(lambda *a: f(*a))(*batched))
        assert isinstance(fast, tuple) and fast[0] is RuntimeError and fast == slow, (fast, slow)
        one = torch.ones((), device=o.x.device)
        for e in _both(monkeypatch, lambda: torch.func.grad(in_grad)(one)):
            assert isinstance(e, tuple) and issubclass(e[0], RuntimeError), e
        f(*args)                                          # and plain tensors as before


def test_outputs_are_what_torch_makes():
    """Each output has a storage of its own from torch's allocator: it grows in
    place without its siblings, knows its streams, and its memory is counted."""
    o = Operands()
    say("calls: outputs like torch's")
    layer = gq.gq_moe_layer(o.router, o.bank, o.down, 2)
    gq.gq_moe_decode(layer, o.x)
    q = gq.gq_mxfp4_quantize(o.x)
    route = gq.gq_route_sort(o.ids, 4)
    ids, w = gq.gq_moe_topk(o.z, 2)
    for f in (lambda: gq.gq_mxfp4_quantize(o.x, values=True), lambda: gq.gq_moe_topk(o.z, 2),
              lambda: gq.gq_route_sort(o.ids, 4)[:4],
              lambda: (gq.gq_moe_topk_backward(w, o.z, ids),),
              lambda: (gq.gq_moe_decode(layer, o.x),),
              lambda: (gq.gq_mxfp4_grouped_gemv_fp4(q, *o.bank, o.ids),),
              lambda: (gq.gq_mxfp4_grouped_gemm_fp4(q, *o.bank, route),)):
        before = torch.cuda.memory_allocated()
        outs = f()
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() > before
        for t in outs:
            like = torch.empty(t.shape, dtype=t.dtype, device=t.device)
            assert torch._C._dispatch_keys(t) == torch._C._dispatch_keys(like)
            assert t.device == like.device and t.stride() == like.stride() and t._version == 0
            assert t.untyped_storage().nbytes() == t.numel() * t.element_size()
            t.record_stream(torch.cuda.Stream())
        kept = [t.clone() for t in outs]
        for i, t in enumerate(outs):
            t.resize_(1 << 16).zero_()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in list(zip(outs, kept))[i + 1:])
        del outs, t, like, kept
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() == before
