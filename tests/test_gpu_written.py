"""Every output of the norm, its gradient, the routing, its gradient and the products
of quantised activations is written: buffers that hold NaN before the call, compared
with float64 in a way that no NaN passes, over every kernel that sizes choose."""

import numpy as np
import pytest
import torch

import bit_grouped_moe_amd as gq
import oracle
import workloads as wl
from tests import test_gpu_fp4 as fp4
from tests import test_gpu_fp8 as fp8
from tests import test_gpu_moe_route as mr
from tests import test_gpu_norm as nm
from tests.gpu_common import LazyDecoded, device, packed_mx_bank, say, to_dev
from tests.strict import assert_within

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _nan(shape, dtype):
    return torch.full(tuple(shape), NAN, dtype=dtype, device="cuda")


def _rounded(want, room, dtype):
    """How far one rounding to the type of a value that is off by `room` may be."""
    rel, least = nm._half(dtype)
    return rel * (want.abs() + room) + room + least


# Rows x widths of each of the norm's forms: 1, 4 and 16 waves a row with one to four
# steps, for up to and over 256 rows, whole and broken 8-value pieces.
NORMS = [(3, 480), (259, 481), (5, 1000), (260, 992), (261, 2048), (9, 1999), (7, 8192),
         (4, 2081), (258, 4096), (259, 3969), (257, 8160), (6, 16384), (3, 9001), (2, 32768),
         (5, 16393)]


@pytest.mark.parametrize("dtype,wtype", nm.TYPES)
@pytest.mark.parametrize("rows,H", NORMS)
def test_norm(dtype, wtype, rows, H):
    dev = device()
    x, r, w = nm._inputs(rows, H, dtype, wtype, seed=3)
    xd, rd, wd = x.to(dev), r.to(dev), w.to(dev)
    q = H % 32 == 0
    pair = (torch.full((rows, H), 0x7F, dtype=torch.uint8, device=dev),
            torch.full((rows, H // 32), 255, dtype=torch.uint8, device=dev)) if q else False
    values = _nan((rows, H), torch.bfloat16) if q else False
    say("norm written", dtype, wtype, rows, H)
    got = gq.gq_rms_norm(xd, wd, eps=1e-5, residual=rd, y=_nan(x.shape, dtype),
                         sum=_nan(x.shape, dtype), mxfp8=pair, values=values)
    dx, dw = gq.gq_rms_norm_backward(
        rd, got.residual, wd, eps=1e-5, d_residual=xd, d_x=_nan(x.shape, dtype),
        d_weight=_nan(w.shape, wtype),
        workspace=torch.full((gq.gq_rms_norm_backward_workspace(rows, H),), 255, dtype=torch.uint8,
                             device=dev))
    torch.cuda.synchronize()
    h = nm._sum(x, r)
    assert torch.equal(got.residual.cpu(), h)
    want = nm._norm(h, w, 1e-5)
    assert_within(got.y, want, _rounded(want, nm.NORM * want.abs(), dtype), "y")
    if q:
        assert torch.isfinite(got.values).all()
        nm._values_are_nearest(*got.mxfp8, got.values, want)
    wx, room, ws, wabs = nm._backward(r, h, w, x, 1e-5)
    assert_within(dx, wx, _rounded(wx, room, dtype), "dx")
    # a lane's rows, the waves of a workgroup and the workgroups' sums, at most
    deep = (rows + 511) // 512 + 4 + 8 + 4 + 16 + 3
    assert_within(dw, ws, _rounded(ws, (deep * nm.U + nm.NORM) * wabs, wtype), "dw")


def _product_room(ref, m):
    return m.ROUND * np.abs(ref) + m.SUMS * np.sqrt((ref ** 2).mean(axis=1, keepdims=True))


# Sizes of experts' segments on both sides of every count of 32-row sub-tiles
SIZES = [1, 32, 33, 64, 97, 128, 129, 160, 193, 224, 225, 256, 257, 300, 0]


@pytest.mark.parametrize("unit", [False, True])
@pytest.mark.parametrize("m,name", [(fp4, "fp4"), (fp8, "fp8")])
@pytest.mark.parametrize("N,K", [(64, 32), (288, 160), (320, 672), (96, 1056), (1312, 96),
                                 (1312, 256), (1312, 416), (2336, 1056)])
def test_product(N, K, m, name, unit):
    """Column tiles of 128 and 256, few and many rows a tile, every tail of K."""
    dev = device()
    g = np.random.default_rng(N + K)
    E = len(SIZES)
    ids = np.concatenate([np.full(n, e, dtype=np.int32) for e, n in enumerate(SIZES)]
                         + [np.full(5, -1, dtype=np.int32), np.full(4, E, dtype=np.int32)])
    ids = g.permutation(ids).reshape(-1, 1)
    P = ids.shape[0]
    bank = packed_mx_bank(g, E, N, K)
    x, xv = m._x(g, P, K)
    ref = m._ref(xv, LazyDecoded("mx", *bank), ids, E, N)
    route = gq.gq_route_sort(to_dev(ids, dev), E)
    args = (m._both(x, dev), *m._both(bank, dev), route)
    out = _nan((P, N // 2 if unit else N), torch.bfloat16)
    say("product written", name, N, K, unit)
    call = getattr(gq, f"gq_mxfp4_grouped_gemm_{name}" + ("_swiglu" if unit else ""))
    call(*args, out=out)
    torch.cuda.synchronize()
    live = (ids >= 0) & (ids < E)
    if unit:
        ref = oracle.swiglu_oss(ref) * live
    assert_within(out, ref, _product_room(ref, m))
    assert not out.cpu()[torch.from_numpy(~live[:, 0])].any()


@pytest.mark.parametrize("unit", [False, True])
@pytest.mark.parametrize("m,name", [(fp4, "fp4"), (fp8, "fp8")])
@pytest.mark.parametrize("rows,topk,E,N,K", [(1, 4, 32, 320, 2880), (8, 4, 6, 96, 256),
                                             (64, 4, 4, 250, 1056), (64, 4, 4, 130, 1056),
                                             (64, 4, 4, 42, 2080), (64, 4, 4, 20, 2080),
                                             (16, 4, 5, 64, 8192), (16, 4, 5, 32, 8192)])
def test_single_token_product(rows, topk, E, N, K, m, name, unit):
    dev = device()
    g = np.random.default_rng(rows + N + K)
    bank = packed_mx_bank(g, E, N, K)
    ids = wl.route_uniform(g, rows, E, topk)
    if rows > 1:
        ids[1, 0], ids[-1, -1] = -1, E
    x, xv = m._x(g, rows, K)
    ref = m._ref(xv, LazyDecoded("mx", *bank), ids, E, N)
    out = _nan((rows * topk, N // 2 if unit else N), torch.bfloat16)
    say("single-token product written", name, rows, N, K, unit)
    call = getattr(gq, f"gq_mxfp4_grouped_gemv_{name}" + ("_swiglu" if unit else ""))
    call(m._both(x, dev), *m._both(bank, dev), to_dev(ids, dev), out=out)
    torch.cuda.synchronize()
    live = ((ids >= 0) & (ids < E)).reshape(-1, 1)
    if unit:
        ref = oracle.swiglu_oss(ref) * live
    assert_within(out, ref, _product_room(ref, m))
    assert not out.cpu()[torch.from_numpy(~live[:, 0])].any()


# A wave and sixteen lanes a row, every width of each, with and without groups.
ROUTES = [(3, 60, 1, 1, 6), (70, 128, 8, 3, 8), (9, 256, 8, 4, 8), (130, 512, 8, 4, 12),
          (5, 1000, 10, 3, 33), (4100, 64, 16, 5, 9), (4097, 128, 1, 1, 8), (2050, 256, 8, 4, 8),
          (4099, 200, 1, 1, 16), (4098, 1024, 1, 1, 64)]


@pytest.mark.parametrize("dtype", mr.DTYPES)
@pytest.mark.parametrize("rows,E,groups,topk_groups,topk", ROUTES)
def test_routing(rows, E, groups, topk_groups, topk, dtype):
    dev = device()
    g = torch.Generator().manual_seed(E + rows)
    for n, (score, kind, bias, renorm) in enumerate((
            ("sigmoid", "random", "random", True), ("sigmoid", "masked", None, False),
            ("softmax", "masked", "random", True), ("softmax", "random", None, False))):
        z, b = mr._logits(g, rows, E, dtype, kind), mr._bias(g, E, bias)
        dw = torch.randn(rows, topk, generator=g)
        ids = torch.full((rows, topk), 99, dtype=torch.int32, device=dev)
        kw = dict(score=score, renormalize=renorm, scale=2.5)
        say("routing written", rows, E, groups, topk, dtype, score, kind, bias)
        _, w = gq.gq_moe_route(
            z.to(dev), topk, bias=None if b is None else b.to(dev), groups=groups,
            topk_groups=topk_groups, group_top=1 + n % 2 if groups > 1 else 1, topk_ids=ids,
            topk_weights=_nan((rows, topk), torch.float32), **kw)
        dz = gq.gq_moe_route_backward(dw.to(dev), z.to(dev), ids, out=_nan(z.shape, dtype), **kw)
        torch.cuda.synchronize()
        zn, at = z.float().numpy(), ids.cpu().numpy()
        assert np.array_equal(at, mr._select(zn, topk, score, None if b is None else b.numpy(),
                                             groups, topk_groups,
                                             1 + n % 2 if groups > 1 else 1))
        want, zs = mr._weights(zn, at, score, renorm, 2.5)
        live = zn[zn > -mr.INF]
        top = np.abs(live).max() if live.size else 0
        # an exponential of a rounded difference to an ulp, the sum's 22 additions, two
        # divisions and two products
        far = np.abs(np.where(np.isfinite(zs), zs, 0)) + top
        assert_within(w, want, (2 * far + 40) * mr.U * np.abs(want) + 2.0 ** -126, "weights")
        want, room = mr._grad(zn, at, dw.numpy(), score, renorm, 2.5)
        # as a weight's rounding, twice (the slot's and the sum's), then the type's
        room = room * (8 * top + 200) * mr.U
        least = {torch.float16: 2.0 ** -25}.get(dtype, 2.0 ** -125)
        assert_within(dz, want, torch.finfo(dtype).eps / 2 * (np.abs(want) + room) + room + least,
                      "d_logits")
