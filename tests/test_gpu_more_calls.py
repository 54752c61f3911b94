"""The two ways to the library, short calls and Python code, of the norm, the
8-bit quantiser and products and the routing with groups: the same outputs, the
same refusals, and outputs that are what torch makes."""

import numpy as np
import pytest
import torch

import bit_grouped_moe_amd as gq
import workloads as wl
from tests.gpu_common import device, packed_mx_bank, say, to_dev, to_dev_bf16
from tests.test_gpu_calls import _both, _same

pytestmark = pytest.mark.gpu


class Operands:
    def __init__(self):
        dev = device()
        g = np.random.default_rng(8)
        self.x = to_dev_bf16(wl.draw_bf16(g, (6, 96)), dev)
        self.r = to_dev_bf16(wl.draw_bf16(g, (6, 96)), dev)
        self.gain = torch.rand(96, device=dev) + 0.5
        self.bank = tuple(to_dev(t, dev) for t in packed_mx_bank(g, 4, 64, 96))
        self.down = tuple(to_dev(t, dev) for t in packed_mx_bank(g, 4, 96, 32))
        self.ids = to_dev(wl.route_uniform(g, 6, 4, 2), dev)
        self.z = torch.from_numpy(g.standard_normal((6, 8)).astype(np.float32)).to(dev)
        self.bias = torch.rand(8, device=dev)
        self.w = torch.rand(12, device=dev)
        self.wide = to_dev_bf16(wl.draw_bf16(g, (6, 200)), dev)


def test_same_outputs(monkeypatch):
    o = Operands()
    say("more calls: outputs")
    q = gq.gq_mxfp8_quantize(o.x)
    route = gq.gq_route_sort(o.ids, 4)
    cut = o.wide[:, 5:101]
    dw = o.w.reshape(6, 2)
    for f in (lambda: gq.gq_mxfp8_quantize(o.x), lambda: gq.gq_mxfp8_quantize(o.x, values=True),
              lambda: gq.gq_mxfp8_quantize(cut.half()), lambda: gq.gq_mxfp8_quantize(cut),
              lambda: gq.gq_mxfp8_quantize(o.x[0]), lambda: gq.gq_mxfp8_quantize(o.x[:0]),
              lambda: gq.gq_mxfp8_quantize(o.x.float().reshape(2, 3, 96), values=True),
              lambda: gq.gq_rms_norm(o.x, o.gain), lambda: gq.gq_rms_norm(o.x, o.gain.bfloat16()),
              lambda: gq.gq_rms_norm(o.x, o.gain, 1e-3, o.r),
              lambda: gq.gq_rms_norm(cut, o.gain, residual=o.wide[:, 7:103], mxfp8=True),
              lambda: gq.gq_rms_norm(o.x, o.gain, residual=cut, mxfp8=True, values=True),
              lambda: gq.gq_rms_norm(o.x[:, :95], o.gain[:95]), lambda: gq.gq_rms_norm(o.x[2], o.gain),
              lambda: gq.gq_rms_norm(o.x.reshape(2, 3, 96), o.gain, residual=o.r.reshape(2, 3, 96)),
              lambda: gq.gq_rms_norm(o.x[:0], o.gain), lambda: gq.gq_rms_norm(cut[:1], o.gain),
              lambda: gq.gq_rms_norm_backward(o.r, o.x, o.gain),
              lambda: gq.gq_rms_norm_backward(cut, o.x, o.gain, 1e-3, o.r),
              lambda: gq.gq_rms_norm_backward(o.r, cut, o.gain.bfloat16(), d_weight=False),
              lambda: gq.gq_rms_norm_backward(o.r[:0], o.x[:0], o.gain),
              lambda: gq.gq_moe_route(o.z, 2), lambda: gq.gq_moe_route(o.z.half(), 3, "sigmoid"),
              lambda: gq.gq_moe_route(o.z, 3, "sigmoid", o.bias, 4, 2, 2, False, 2.5),
              lambda: gq.gq_moe_route(o.z, 2, groups=2), lambda: gq.gq_moe_route(o.z[:, 1:7], 2),
              lambda: gq.gq_moe_route(o.z[:0], 2), lambda: gq.gq_moe_route(o.z, 2, scale=2),
              lambda: gq.gq_moe_route_backward(dw, o.z, o.ids),
              lambda: gq.gq_moe_route_backward(dw, o.z.bfloat16(), o.ids, "sigmoid", False, 3),
              lambda: gq.gq_mxfp4_grouped_gemv_fp8(q, *o.bank, o.ids),
              lambda: gq.gq_mxfp4_grouped_gemv_fp8(q, *o.bank, o.ids, pair_scale=o.w),
              lambda: gq.gq_mxfp4_grouped_gemv_fp8_swiglu(q, *o.bank, o.ids, limit=2.0),
              lambda: gq.gq_mxfp4_grouped_gemm_fp8(q, *o.bank, route),
              lambda: gq.gq_mxfp4_grouped_gemm_fp8(q, *o.bank, route, pair_scale=o.w),
              lambda: gq.gq_mxfp4_grouped_gemm_fp8_swiglu(q, *o.bank, route, alpha=1, limit=3)):
        fast, slow = _both(monkeypatch, f)
        assert not (isinstance(fast, tuple) and isinstance(fast[0], type)), fast
        _same(fast, slow)


def test_same_refusals(monkeypatch):
    o = Operands()
    say("more calls: refusals")
    q = gq.gq_mxfp8_quantize(o.x)
    q4 = gq.gq_mxfp4_quantize(o.x)
    route = gq.gq_route_sort(o.ids, 4)
    cpu, nan = o.x.cpu(), float("nan")
    dw = o.w.reshape(6, 2)
    for f in (lambda: gq.gq_mxfp8_quantize(cpu), lambda: gq.gq_mxfp8_quantize(None),
              lambda: gq.gq_mxfp8_quantize(o.x[:, :40]), lambda: gq.gq_mxfp8_quantize(o.x[:, ::2]),
              lambda: gq.gq_mxfp8_quantize(o.ids), lambda: gq.gq_mxfp8_quantize(o.x.t()),
              lambda: gq.gq_mxfp8_quantize(o.x[:1].expand(6, 96)),
              lambda: gq.gq_rms_norm(cpu, o.gain), lambda: gq.gq_rms_norm(o.x, o.gain.cpu()),
              lambda: gq.gq_rms_norm(o.x, o.gain[:95]), lambda: gq.gq_rms_norm(o.x, o.gain.half()),
              lambda: gq.gq_rms_norm(o.x, o.gain.repeat(2)[::2]), lambda: gq.gq_rms_norm(o.x, 1.0),
              lambda: gq.gq_rms_norm(o.x, o.gain, -1.0), lambda: gq.gq_rms_norm(o.x, o.gain, nan),
              lambda: gq.gq_rms_norm(o.x, o.gain, "x"), lambda: gq.gq_rms_norm(o.x, o.gain, None),
              lambda: gq.gq_rms_norm(o.x, o.gain, residual=o.r[:3]),
              lambda: gq.gq_rms_norm(o.x, o.gain, residual=o.r.float()),
              lambda: gq.gq_rms_norm(o.x, o.gain, residual=o.r[:1].expand(6, 96)),
              lambda: gq.gq_rms_norm(o.x[:1].expand(6, 96), o.gain),
              lambda: gq.gq_rms_norm(o.x[:, :95], o.gain[:95], mxfp8=True),
              lambda: gq.gq_rms_norm(o.x, o.gain, values=True), lambda: gq.gq_rms_norm(o.ids, o.gain),
              lambda: gq.gq_rms_norm(o.wide[:, ::2][:, :96], o.gain),
              lambda: gq.gq_rms_norm(torch.zeros(2, 40000, device=o.x.device),
                                     torch.zeros(40000, device=o.x.device)),
              lambda: gq.gq_rms_norm_backward(o.r[:3], o.x, o.gain),
              lambda: gq.gq_rms_norm_backward(None, o.x, o.gain),
              lambda: gq.gq_rms_norm_backward(o.r, o.x, o.gain, d_residual=o.r.half()),
              lambda: gq.gq_rms_norm_backward(o.r, o.x, o.gain, -1.0),
              lambda: gq.gq_rms_norm_backward(torch.zeros(2, 40000, device=o.x.device),
                                              torch.zeros(2, 40000, device=o.x.device),
                                              torch.zeros(40000, device=o.x.device)),
              lambda: gq.gq_moe_route(o.z, 0), lambda: gq.gq_moe_route(o.z, 9),
              lambda: gq.gq_moe_route(o.z, 1 << 70), lambda: gq.gq_moe_route(o.z, 2, "relu"),
              lambda: gq.gq_moe_route(o.z, 2, bias=o.bias[:7]),
              lambda: gq.gq_moe_route(o.z, 2, bias=o.bias.half()),
              lambda: gq.gq_moe_route(o.z, 2, groups=3), lambda: gq.gq_moe_route(o.z, 2, groups=0),
              lambda: gq.gq_moe_route(o.z, 2, groups=4, topk_groups=5),
              lambda: gq.gq_moe_route(o.z, 2, groups=4, topk_groups=0),
              lambda: gq.gq_moe_route(o.z, 3, groups=4, topk_groups=1),
              lambda: gq.gq_moe_route(o.z, 2, groups=4, topk_groups=1 << 40),
              lambda: gq.gq_moe_route(o.z, 2, group_top=3), lambda: gq.gq_moe_route(o.z, 2, scale=nan),
              lambda: gq.gq_moe_route(o.z, 2, scale="x"), lambda: gq.gq_moe_route(o.z[0], 2),
              lambda: gq.gq_moe_route(o.z.double(), 2),
              lambda: gq.gq_moe_route_backward(o.w, o.z, o.ids),
              lambda: gq.gq_moe_route_backward(dw, o.z, o.ids.long()),
              lambda: gq.gq_moe_route_backward(dw, o.z, o.ids, "relu"),
              lambda: gq.gq_moe_route_backward(dw, o.z, o.ids, scale=nan),
              lambda: gq.gq_mxfp4_grouped_gemv_fp8(q4, *o.bank, o.ids),
              lambda: gq.gq_mxfp4_grouped_gemv_fp4(q, *o.bank, o.ids),
              lambda: gq.gq_mxfp4_grouped_gemv_fp8(q, *o.bank, o.ids[:4]),
              lambda: gq.gq_mxfp4_grouped_gemv_fp8(q, *o.bank, o.ids, pair_scale=o.w[:3]),
              lambda: gq.gq_mxfp4_grouped_gemv_fp8_swiglu(q, *o.bank, o.ids, alpha=nan),
              lambda: gq.gq_mxfp4_grouped_gemm_fp8(q4, *o.bank, route),
              lambda: gq.gq_mxfp4_grouped_gemm_fp8(q, *o.down, route),
              lambda: gq.gq_mxfp4_grouped_gemm_fp8(q, *o.bank, route._replace(tile_m=128)),
              lambda: gq.gq_mxfp4_grouped_gemm_fp8(q, *o.bank, route._replace(max_tiles=1)),
              lambda: gq.gq_mxfp4_grouped_gemm_fp8(q, *o.bank, route._replace(topk=3)),
              lambda: gq.gq_mxfp4_grouped_gemm_fp8_swiglu(q, *o.bank, route, limit=-1.0)):
        fast, slow = _both(monkeypatch, f)
        assert isinstance(fast, tuple) and isinstance(fast[0], type), fast
        assert fast == slow


def test_outputs_are_what_torch_makes():
    """Each output has a storage of its own from torch's allocator."""
    o = Operands()
    say("more calls: outputs like torch's")
    q = gq.gq_mxfp8_quantize(o.x)
    route = gq.gq_route_sort(o.ids, 4)
    dw = o.w.reshape(6, 2)

    def flat(n):
        return (n.y, n.residual, *n.mxfp8, n.values)

    for f in (lambda: gq.gq_mxfp8_quantize(o.x, values=True),
              lambda: flat(gq.gq_rms_norm(o.x, o.gain, residual=o.r, mxfp8=True, values=True)),
              lambda: gq.gq_rms_norm_backward(o.r, o.x, o.gain),
              lambda: gq.gq_moe_route(o.z, 2, "sigmoid", o.bias),
              lambda: (gq.gq_moe_route_backward(dw, o.z, o.ids),),
              lambda: (gq.gq_mxfp4_grouped_gemv_fp8(q, *o.bank, o.ids),),
              lambda: (gq.gq_mxfp4_grouped_gemm_fp8(q, *o.bank, route),)):
        before = torch.cuda.memory_allocated()
        outs = f()
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() > before
        for t in outs:
            like = torch.empty(t.shape, dtype=t.dtype, device=t.device)
            assert torch._C._dispatch_keys(t) == torch._C._dispatch_keys(like)
            assert t.device == like.device and t.stride() == like.stride() and t._version == 0
            assert t.untyped_storage().nbytes() == t.numel() * t.element_size()
            assert not t.requires_grad and t.is_leaf
        kept = [t.clone() for t in outs]
        for i, t in enumerate(outs):
            t.resize_(1 << 16).zero_()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in list(zip(outs, kept))[i + 1:])
        del outs, t, like, kept
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() == before


def test_a_stream_of_its_own():
    o = Operands()
    say("more calls: side stream")
    x = torch.randn(4096, 2880, device=o.x.device).to(torch.bfloat16)
    gain = torch.rand(2880, device=x.device)
    ref = gq.gq_rms_norm(x, gain, residual=x, mxfp8=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = x * 0.5
        y = y * 2                                          # on s, before the call
        got = gq.gq_rms_norm(y, gain, residual=x, mxfp8=True)
        dx, dw = gq.gq_rms_norm_backward(got.y, got.residual, gain)
    s.synchronize()
    _same(got, ref)
    _same((dx, dw), gq.gq_rms_norm_backward(ref.y, ref.residual, gain))


def test_two_streams_at_once():
    """Calls in flight on two streams, workspaces and outputs of their own: the
    bytes of the same calls one after the other."""
    dev = device()
    g = torch.Generator().manual_seed(31)
    E, H, N, rows = 6, 512, 320, 700
    w = torch.rand(H, generator=g).to(torch.bfloat16).to(dev)
    blocks = torch.randint(0, 256, (E, N, H // 32, 16), dtype=torch.uint8, generator=g).to(dev)
    scales = torch.randint(120, 128, (E, N, H // 32), dtype=torch.uint8, generator=g).to(dev)
    bias = (0.1 * torch.randn(E, generator=g)).to(dev)
    sets = [[torch.randn(rows, n, generator=g).to(torch.bfloat16).to(dev) for n in (H, H, H, E)]
            for _ in range(2)]

    def block(x, r, dy, z):
        n = gq.gq_rms_norm(x, w, residual=r, mxfp8=True)
        ids, weights = gq.gq_moe_route(z, 2, score="sigmoid", bias=bias, groups=3, topk_groups=2)
        y = gq.gq_mxfp4_grouped_gemm_fp8(n.mxfp8, blocks, scales, gq.gq_route_sort(ids, E),
                                         pair_scale=weights.reshape(-1))
        dx, dw = gq.gq_rms_norm_backward(dy, n.residual, w, d_residual=x)
        dz = gq.gq_moe_route_backward(weights, z, ids, score="sigmoid")
        return n.y, *n.mxfp8, ids, weights, y, dx, dw, dz

    say("two streams")
    want = [block(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(block(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for one in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(one, want[i]))
