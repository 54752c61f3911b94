"""Expert routing on the GPU against its definition in float64: the chosen
experts exactly, weights and gradients to float32 rounding."""

import numpy as np
import pytest
import torch

import bit_grouped_moe_amd as gq
from tests.gpu_common import device, say

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
U = 2.0 ** -24                                  # half a float32 step


def _select(z, topk):
    """Ids by a stable sort of the float64 logits (-inf never chosen)."""
    order = np.argsort(-z, axis=1, kind="stable")[:, :topk]
    live = np.take_along_axis(z, order, 1) > -np.inf
    return np.where(live, order, -1)


def _weights(z, ids, renorm):
    """float64 weights of given slots."""
    rows, E = z.shape
    ok = (ids >= 0) & (ids < E)
    zs = np.where(ok, np.take_along_axis(z, np.clip(ids, 0, E - 1), 1), -np.inf)
    pool = zs if renorm else z
    peak = pool.max(axis=1, keepdims=True)
    peak = np.where(np.isfinite(peak), peak, 0.0)
    total = np.exp(pool - peak).sum(axis=1, keepdims=True)
    return np.exp(zs - peak) / np.where(total > 0, total, 1.0), peak - zs


def _grad(z, ids, dw, renorm):
    """The softmax Jacobian applied slot by slot, float64."""
    rows, E = z.shape
    w, _ = _weights(z, ids, renorm)
    out = np.zeros_like(z)
    for r in range(rows):
        for s in range(ids.shape[1]):
            j = ids[r, s]
            if not 0 <= j < E or w[r, s] == 0:
                continue
            out[r, j] += dw[r, s] * w[r, s]
            if renorm:
                for q in range(ids.shape[1]):
                    if 0 <= ids[r, q] < E:
                        out[r, ids[r, q]] -= dw[r, s] * w[r, s] * w[r, q]
            else:
                peak = z[r].max()
                p = np.exp(z[r] - peak)
                out[r] -= dw[r, s] * w[r, s] * p / p.sum()
    return out


def _logits(g, rows, E, dtype, kind):
    z = torch.randn(rows, E, generator=g) * 3
    if kind == "ties":
        z = (z * 2).round() / 2
        z[z == 0] = -0.0
        z[:, ::2][z[:, ::2] == 0] = 0.0                  # -0 and +0 are equal
    if kind == "masked":
        z[torch.rand(rows, E, generator=g) < 0.5] = -float("inf")
        z[0] = -float("inf")
        if rows > 1:
            z[1] = torch.finfo(dtype).min                # the lowest value is a value
    return z.to(dtype)


def _check_forward(z, ids, w, topk, renorm):
    z64 = z.double().cpu().numpy()
    ref = _select(z64, topk)
    assert np.array_equal(ids.cpu().numpy(), ref)
    rw, gap = _weights(z64, ref, renorm)
    # the exponent's argument is off by half a step of its size, exp, sum
    # (at most 16 + 6 additions) and quotient by a few steps more
    tol = (np.where(np.isfinite(gap), np.abs(gap), 0) + 40) * U * rw + 1e-37
    assert (np.abs(w.double().cpu().numpy() - rw) <= tol).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["plain", "ties", "masked"])
@pytest.mark.parametrize("rows,E,topk", [(1, 1, 1), (1, 128, 8), (7, 5, 5), (33, 32, 4),
                                         (5, 64, 64), (6, 65, 3), (130, 129, 8), (9, 300, 10),
                                         (4, 512, 2), (3, 1024, 33)])
def test_forward_and_backward(dtype, kind, rows, E, topk):
    dev = device()
    g = torch.Generator().manual_seed(rows * 1000 + E + topk)
    z = _logits(g, rows, E, dtype, kind)
    dw = torch.randn(rows, topk, generator=g)
    zd, dwd = z.to(dev), dw.to(dev)
    for renorm in (True, False):
        say("router", dtype, kind, rows, E, topk, renorm)
        ids, w = gq.gq_moe_topk(zd, topk, renormalize=renorm)
        dz = gq.gq_moe_topk_backward(dwd, zd, ids, renormalize=renorm)
        torch.cuda.synchronize()
        _check_forward(z, ids, w, topk, renorm)
        assert dz.dtype == dtype and dz.shape == z.shape
        z64, d64, i64 = z.double().numpy(), dw.double().numpy(), ids.cpu().numpy()
        ref = _grad(z64, i64, d64, renorm)
        w64, gap = _weights(z64, i64, renorm)
        # each term p (g - sum p g) at the rounding of p, one product and a
        # sum of at most 64 slots; then one rounding to the output's type
        big = (np.abs(d64).max(axis=1) * 2)[:, None]
        pool = np.where(np.isfinite(z64), z64, -np.inf)
        peak = pool.max(axis=1, keepdims=True)
        p = np.where(np.isfinite(peak), np.exp(pool - np.where(np.isfinite(peak), peak, 0)), 0)
        p = p / np.maximum(p.sum(axis=1, keepdims=True), 1e-300)
        if renorm:                                       # chosen experts only, larger weights
            p = np.zeros_like(p)
            for r in range(rows):
                for s in range(topk):
                    if i64[r, s] >= 0:
                        p[r, i64[r, s]] += w64[r, s]
        spread = np.where(np.isfinite(z64), np.abs(peak - z64), 0)
        spread = np.where(np.isfinite(spread) & (p > 0), spread, 0)
        tol = p * big * (spread + 120) * U
        # (below its normal range an output type has a fixed step)
        tol = tol + np.abs(ref) * torch.finfo(dtype).eps / 2 + (
            2.0 ** -25 if dtype == torch.float16 else 1e-37)
        assert (np.abs(dz.double().cpu().numpy() - ref) <= tol * 1.0001).all()


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(renorm):
    """The kernel's gradient against central differences of the float64
    weights, the selection held fixed: truncation h^2 / 6 times the third
    derivative (below 6 for a softmax) and rounding 1e-16 / h."""
    dev = device()
    g = torch.Generator().manual_seed(17)
    rows, E, topk, h = 4, 24, 5, 1e-4
    z = torch.randn(rows, E, generator=g)
    dw = torch.randn(rows, topk, generator=g)
    say("router differences", renorm)
    ids, _ = gq.gq_moe_topk(z.to(dev), topk, renormalize=renorm)
    dz = gq.gq_moe_topk_backward(dw.to(dev), z.to(dev), ids, renormalize=renorm)
    torch.cuda.synchronize()
    z64, i64, d64 = z.double().numpy(), ids.cpu().numpy(), dw.double().numpy()
    num = np.zeros_like(z64)
    for j in range(E):
        up, dn = z64.copy(), z64.copy()
        up[:, j] += h
        dn[:, j] -= h
        num[:, j] = ((_weights(up, i64, renorm)[0] - _weights(dn, i64, renorm)[0]) * d64).sum(
            axis=1) / (2 * h)
    big = np.abs(d64).sum(axis=1, keepdims=True)
    assert (np.abs(dz.double().cpu().numpy() - num) <= big * (h * h + 1e-11 + 200 * U)).all()


@pytest.mark.parametrize("renorm", [True, False])
def test_backward_of_given_ids(renorm):
    """Ids of the caller's own: an expert named twice, ids outside [0, E), a
    masked expert."""
    dev = device()
    z = torch.tensor([[0.5, -1.0, 2.0, -float("inf"), 0.25], [-float("inf")] * 5])
    ids = torch.tensor([[2, 2, -1, 3, 7, 0], [0, 1, 2, 3, 4, -1]], dtype=torch.int32)
    dw = torch.tensor([[1.0, -2.0, 5.0, 7.0, 9.0, 0.5], [1.0] * 6])
    say("router given ids", renorm)
    dz = gq.gq_moe_topk_backward(dw.to(dev), z.to(dev), ids.to(dev), renormalize=renorm)
    torch.cuda.synchronize()
    z64, d64, i64 = z.double().numpy(), dw.double().numpy(), ids.numpy()
    ref = np.zeros((2, 5))
    slots = [(2, 1.0), (2, -2.0), (0, 0.5)]
    if renorm:
        e = np.exp(np.array([z64[0, j] for j, _ in slots]) - 2.0)
        p = e / e.sum()
        dot = sum(pi * d for pi, (_, d) in zip(p, slots))
        for pi, (j, d) in zip(p, slots):
            ref[0, j] += pi * (d - dot)
    else:
        p = np.exp(z64[0] - 2.0)
        p = p / p.sum()
        dot = sum(p[j] * d for j, d in slots)
        G = np.zeros(5)
        for j, d in slots:
            G[j] += d
        ref[0] = p * (G - dot)
    assert np.abs(dz.double().cpu().numpy() - ref).max() <= 100 * U * np.abs(d64).max()
    assert not dz[1].any() and dz[0, 3] == 0


def test_nan_and_infinite_logits_are_not_hidden():
    dev = device()
    nan, inf = float("nan"), float("inf")
    z = torch.tensor([[0.0, nan, 1.0, nan], [inf, 0.0, 1.0, 2.0], [0.0, 1.0, 2.0, 3.0],
                      [-nan, -inf, -inf, -inf]])
    say("router nan")
    ids, w = gq.gq_moe_topk(z.to(dev), 2)
    torch.cuda.synchronize()
    assert ids.tolist() == [[1, 3], [0, 3], [3, 2], [0, -1]]
    w = w.cpu()
    assert w[0].isnan().all() and w[1, 0].isnan() and w[3, 0].isnan() and w[3, 1] == 0
    assert abs(float(w[2].sum()) - 1) < 1e-6


def test_strided_rows_empty_and_large():
    dev = device()
    g = torch.Generator().manual_seed(3)
    z = torch.randn(50, 200, generator=g).to(torch.bfloat16)
    part = z.to(dev)[::2, 3:67]
    say("router strided")
    ids, w = gq.gq_moe_topk(part, 6)
    dz = gq.gq_moe_topk_backward(torch.ones(25, 6, device=dev), part, ids)
    torch.cuda.synchronize()
    _check_forward(z[::2, 3:67], ids, w, 6, True)
    assert dz.shape == (25, 64)
    # all weights of a row up together: the softmax does not move
    assert float(dz.float().abs().max()) <= 64 * U
    ids, w = gq.gq_moe_topk(part[:0], 6)
    assert ids.shape == (0, 6) and w.shape == (0, 6)
    assert gq.gq_moe_topk_backward(w, part[:0], ids).shape == (0, 64)
    big = torch.randn(100003, 32, generator=g)
    ids, w = gq.gq_moe_topk(big.to(dev), 4, renormalize=False)
    torch.cuda.synchronize()
    _check_forward(big, ids, w, 4, False)
    with pytest.raises(gq.GQError):
        gq.gq_moe_topk(part, 65)
    with pytest.raises(ValueError):
        gq.gq_moe_topk(part, 0)
    with pytest.raises(ValueError):
        gq.gq_moe_topk_backward(w, part, ids)


def test_routing_feeds_the_sort():
    """Slots without an expert become dropped pairs of the grouping."""
    dev = device()
    z = torch.randn(70, 16, generator=torch.Generator().manual_seed(4))
    z[::5] = -float("inf")
    z[1::5, 1:] = -float("inf")
    say("router into sort")
    ids, w = gq.gq_moe_topk(z.to(dev), 3)
    route = gq.gq_route_sort(ids, 16)
    torch.cuda.synchronize()
    live = int((ids >= 0).sum())
    assert live == 42 * 3 + 14
    assert int(route.expert_offsets[-1]) == live
    assert not w.cpu()[::5].any() and (w.cpu()[1::5, 0] == 1).all()


def _forward_by_hand(z, topk):
    """Ids and float64 weights, one row at a time in plain Python."""
    ids, ws = [], []
    for row in z.double().tolist():
        order = sorted((e for e in range(len(row)) if row[e] > -np.inf), key=lambda e: (-row[e], e))
        mine = order[:topk] + [-1] * (topk - len(order[:topk]))
        top = max((row[e] for e in mine if e >= 0), default=0.0)
        ex = [np.exp(row[e] - top) if e >= 0 else 0.0 for e in mine]
        ids.append(mine)
        ws.append([v / (sum(ex) or 1.0) for v in ex])
    return np.array(ids), np.array(ws)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,topk", [
    (E, k) for k in (1, 15, 16, 17)
    for E in (1, 3, 4, 63, 64, 65, 67, 72, 128, 130, 144, 255, 256, 257, 272) if k <= E])
def test_sizes_where_the_variants_meet(dtype, E, topk):
    """Row counts that end inside a workgroup, rows at every alignment, few
    distinct logits, and the gradient of ids with repeats and holes; with many
    rows a few, the last among them, are compared."""
    dev = device()
    g = torch.Generator().manual_seed(E * 100 + topk)
    for rows, pad, at in ((1, 0, 0), (17, 5, 2), (4095, 0, 0), (4101, 1, 1), (8209, 8, 8),
                          (64 * E + 4096, 0, 0)):
        say("router variants", dtype, E, topk, rows, pad, at)
        z = (torch.randn(rows, E, generator=g) * 2).round() / 2
        z[torch.rand(rows, E, generator=g) < 0.2] = -float("inf")
        room = torch.full((rows, E + pad), float("inf"), dtype=dtype, device=dev)
        zd = room[:, at:at + E]
        zd.copy_(z)
        ids, w = gq.gq_moe_topk(zd, topk)
        torch.cuda.synchronize()
        at = sorted({0, rows // 2, rows - 2, rows - 1} & set(range(rows)))
        rid, rw = _forward_by_hand(z[at], topk)
        assert np.array_equal(ids.cpu().numpy()[at], rid)
        assert (np.abs(w[at].double().cpu().numpy() - rw) <= 60 * U * rw + 1e-37).all()
        order = np.argsort(-z.double().numpy(), axis=1, kind="stable")[:, :topk]
        live = np.isfinite(np.take_along_axis(z.numpy(), order, 1))
        assert np.array_equal(ids.cpu().numpy(), np.where(live, order, -1))
        given = torch.randint(-2, E + 2, (rows, topk), generator=g, dtype=torch.int32)
        dw = torch.randn(rows, topk, generator=g)
        for renorm in (True, False):
            dz = gq.gq_moe_topk_backward(dw.to(dev), zd, given.to(dev), renormalize=renorm)
            torch.cuda.synchronize()
            ref = np.zeros((len(at), E))
            z64, d64 = z[at].double().numpy(), dw[at].double().numpy()
            for r in range(len(at)):
                slots = [(int(j), d64[r, s]) for s, j in enumerate(given[at][r]) if
                         0 <= j < E and z64[r, j] > -np.inf]
                if not slots:
                    continue
                over = [j for j, _ in slots] if renorm else range(E)
                top = max(z64[r, j] for j in over)
                total = sum(np.exp(z64[r, j] - top) for j in over)
                p = np.exp(z64[r] - top) / total
                dot = sum(p[j] * d for j, d in slots)
                if renorm:
                    for j, d in slots:
                        ref[r, j] += p[j] * (d - dot)
                else:
                    G = np.zeros(E)
                    for j, d in slots:
                        G[j] += d
                    ref[r] = p * (G - dot)
            # p <= 1; a slot's gradient, the sum p g and their difference are
            # each below 4 of the largest |dw| a slot; exp, sums of at most 17
            # + 272 terms and the quotient; the type's own rounding
            big = np.abs(d64).max(axis=1, keepdims=True) * topk * 4
            tol = big * 80 * U + np.abs(ref) * torch.finfo(dtype).eps / 2 * 1.0001 + (
                2.0 ** -25 if dtype == torch.float16 else 1e-37)
            assert (np.abs(dz[at].double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("rows,dtype", [(5, torch.float32), (5000, torch.bfloat16)])
def test_replayed_graph(rows, dtype):
    """Selection, grouping and gradient captured once and replayed on new
    logits, with eager calls on other data between the replays."""
    dev = device()
    g = torch.Generator().manual_seed(rows)
    say("router graph", rows, dtype)
    z = torch.randn(rows, 96, generator=g).to(dtype).to(dev)
    dw = torch.randn(rows, 6, generator=g).to(dev)
    other = torch.randn(rows, 96, generator=g).to(dtype).to(dev)

    def step(logits):
        ids, w = gq.gq_moe_topk(logits, 6)
        return (ids, w, gq.gq_moe_topk_backward(dw, logits, ids), *gq.gq_route_sort(ids, 96)[:4])

    step(z)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(z)
    for _ in range(4):
        z.copy_(torch.randn(rows, 96, generator=g).to(dtype))
        ref = [t.clone() for t in step(z)]
        graph.replay()
        step(other)
        torch.cuda.synchronize()
        for a, b in zip(held, ref):
            assert torch.equal(a, b)


def _slices(rows, piece):
    """Row ranges at the start, around the end of each piece and at the end."""
    at = {0, rows - 8192}
    at |= {b - 4096 for b in range(piece, rows, piece) if b + 4096 < rows}
    return [slice(a, a + 8192) for a in sorted(at)]


@pytest.mark.parametrize("E,topk,piece", [(2, 2, (1 << 28) - 16), (17, 17, (1 << 26) - 4)])
def test_more_rows_than_a_launch_takes(E, topk, piece):
    """Sixteen lanes a row and a wave a row, past the workgroups of a launch:
    rows around the joint and the last ones, and no row left out.  (8192 rows
    by themselves take the same variant.)"""
    dev = device()
    rows = piece + 4099
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    say("router many launches", E, topk, rows)
    g = torch.Generator(device=dev).manual_seed(E)
    z = torch.empty(rows, E, dtype=torch.bfloat16, device=dev).normal_(generator=g)
    z[::7] = -float("inf")
    ids = torch.full((rows, topk), -7, dtype=torch.int32, device=dev)
    w = torch.full((rows, topk), -7.0, device=dev)
    gq.gq_moe_topk(z, topk, topk_ids=ids, topk_weights=w)
    dw = torch.empty(rows, topk, device=dev).normal_(generator=g)
    dz = torch.full((rows, E), float("inf"), dtype=torch.bfloat16, device=dev)
    gq.gq_moe_topk_backward(dw, z, ids, renormalize=False, out=dz)
    torch.cuda.synchronize()
    assert int(ids.min()) == -1 and int(ids.max()) == E - 1
    assert float(w.min()) == 0 and float(w.max()) <= 1
    assert float(dz.abs().max()) < 1e3
    for s in _slices(rows, piece):
        say("rows", s)
        i, v = gq.gq_moe_topk(z[s], topk)
        d = gq.gq_moe_topk_backward(dw[s], z[s], i, renormalize=False)
        torch.cuda.synchronize()
        assert torch.equal(i, ids[s]) and torch.equal(v, w[s]) and torch.equal(d, dz[s])
        _check_forward(z[s].cpu(), i, v, topk, True)


def test_sizes_past_32_bits_are_refused():
    dev = device()
    say("router sizes past 32 bits")
    wide = torch.zeros(1, (1 << 32) + 8, dtype=torch.bfloat16, device=dev)
    z = torch.zeros(1, 8, device=dev)
    ids, w = gq.gq_moe_topk(z, 2)
    with pytest.raises(gq.GQError):
        gq.gq_moe_topk(wide, 2)
    with pytest.raises(gq.GQError):
        gq.gq_moe_topk(z, (1 << 32) + 2)
    with pytest.raises(gq.GQError):
        gq.gq_moe_topk_backward(w, wide, ids)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E", [1, 33, 64, 100, 128, 200, 256])
def test_softmax_over_all_experts_in_both_variants(dtype, E):
    """Not renormalised, few rows and many, masked experts among them."""
    dev = device()
    g = torch.Generator().manual_seed(E)
    for rows in (70, 64 * E + 4099):
        z = torch.randn(rows, E, generator=g) * 3
        z[torch.rand(rows, E, generator=g) < 0.3] = -float("inf")
        z[5] = -float("inf")
        z = z.to(dtype)
        say("router softmax over all", dtype, E, rows)
        ids, w = gq.gq_moe_topk(z.to(dev), min(E, 9), renormalize=False)
        torch.cuda.synchronize()
        at = torch.cat([torch.arange(70), torch.arange(rows - 300, rows)]) if rows > 370 else slice(0, rows)
        _check_forward(z[at], ids[at], w[at], min(E, 9), False)
