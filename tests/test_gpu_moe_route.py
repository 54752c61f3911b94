"""Routing with scores of either kind, a balancing bias and groups on the GPU
against its definition in float64: the chosen experts exactly, weights and
gradients to float32 rounding."""

import numpy as np
import pytest
import torch

import bit_grouped_moe_amd as gq
import oracle
import workloads as wl
from tests.gpu_common import (LazyDecoded, bf16_to_host_f32, device, packed_mx_bank, say, to_dev)

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
U = 2.0 ** -24                                  # half a float32 step
INF = float("inf")


def _scores(z, score):
    z = z.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1 / (1 + np.exp(-z))
        peak = z.max(axis=1, keepdims=True)
        p = np.exp(z - np.where(peak == -INF, 0, peak))
        total = p.sum(axis=1, keepdims=True)
        return p / np.where(total == 0, 1, total)


def _order(v):
    """Places of the last axis, largest first, NaN above all, ties to the lower."""
    return np.argsort(np.where(np.isnan(v), -np.inf, -v), axis=-1, kind="stable") if not (
        np.isnan(v).any()) else np.lexsort((np.where(np.isnan(v), 0, -v), ~np.isnan(v)), axis=-1)


def _select(z, topk, score, bias, groups, topk_groups, group_top):
    z = z.astype(np.float64)
    rows, E = z.shape
    s = _scores(z, score)
    c = z if bias is None else s + bias.astype(np.float64)
    c = np.where(z == -INF, -INF, c)
    if groups > 1:
        v = np.where(c == -INF, -INF, s) if bias is None and group_top == 2 else c
        v = v.reshape(rows, groups, -1)
        v = np.take_along_axis(v, _order(v), 2)[..., :group_top]
        first = v[..., 0]
        value = first + np.where(v[..., 1:] == -INF, 0, v[..., 1:]).sum(axis=2)
        value = np.where(first == -INF, -INF, value)
        keep = np.zeros((rows, groups), dtype=bool)
        np.put_along_axis(keep, _order(value)[:, :topk_groups], True, 1)
        c = np.where(np.repeat(keep, E // groups, axis=1), c, -INF)
    ids = _order(c)[:, :topk]
    return np.where(np.take_along_axis(c, ids, 1) == -INF, -1, ids)


def _weights(z, ids, score, renorm, scale):
    """float64 weights of given slots, through logarithms (no underflow)."""
    z = z.astype(np.float64)
    live = (ids >= 0) & (ids < z.shape[1])
    zs = np.where(live, np.take_along_axis(z, np.clip(ids, 0, z.shape[1] - 1), 1), -INF)
    with np.errstate(invalid="ignore"):
        if score == "sigmoid":
            lw = np.where(zs == -INF, -INF, -np.logaddexp(0, -zs))
        else:
            peak = z.max(axis=1, keepdims=True)
            peak = np.where(peak == -INF, 0, peak)
            lw = zs - peak - np.log(np.maximum(np.exp(z - peak).sum(axis=1, keepdims=True), 1e-300))
        if renorm:
            peak = lw.max(axis=1, keepdims=True)
            peak = np.where(peak == -INF, 0, peak)
            total = np.exp(lw - peak).sum(axis=1, keepdims=True)
            lw = lw - peak - np.log(np.where(total == 0, 1, total))
        return np.exp(lw) * scale, zs


def _check_weights(got, z, ids, score, renorm, scale):
    want, zs = _weights(z, ids, score, renorm, scale)
    zf = np.where(np.isfinite(zs), zs, 0)
    live = z[z > -INF]
    far = np.abs(zf) + (np.abs(live).max() if live.size else 0)
    # an exponential of a rounded difference (its size times U) to an ulp, at most
    # 16 added in a lane and 6 levels of lanes, two divisions and two products
    room = (2 * far + 40) * U
    bad = np.abs(got.cpu().numpy().astype(np.float64) - want) > room * np.abs(want) + 2.0 ** -126
    assert not bad.any(), np.argwhere(bad)[:6].tolist()


def _logits(g, rows, E, dtype, kind):
    z = torch.randn(rows, E, generator=g) * 2
    if kind == "ties":
        z = (z * 2).round() / 2
    elif kind == "masked":
        z[torch.rand(rows, E, generator=g) < 0.5] = -INF
        z[::5] = -INF
    elif kind == "low":                         # every score underflows a float32
        z = z * 5 - 200
    return z.to(dtype)


def _bias(g, E, kind):
    if kind is None:
        return None
    b = torch.randn(E, generator=g) * 0.2
    if kind == "zero":
        b.zero_()
    elif kind == "off":                         # experts that are switched off
        b[torch.rand(E, generator=g) < 0.3] = -INF
    return b


SHAPES = [  # E, groups, topk_groups, topk
    (1, 1, 1, 1), (5, 1, 1, 5), (8, 4, 2, 3), (60, 6, 3, 6), (64, 8, 8, 64), (65, 13, 4, 7),
    (128, 1, 1, 8), (160, 8, 3, 6), (256, 8, 4, 8), (256, 16, 1, 16), (252, 4, 3, 9),
    (320, 64, 20, 10), (512, 8, 4, 12), (1000, 10, 3, 33), (1024, 1, 1, 64), (1024, 64, 7, 17),
    (96, 48, 5, 10), (40, 40, 11, 9)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,topk_groups,topk", SHAPES)
def test_routes(E, groups, topk_groups, topk, score):
    dev = device()
    g = torch.Generator().manual_seed(E + 31 * groups + topk)
    n = 0
    for dtype in DTYPES:
        for kind in ("random", "ties", "masked", "low"):
            for bk in (None, "random", "zero", "off"):
                for top in ((1, 2) if groups > 1 else (1,)):
                    n += 1
                    renorm, scale = n % 2 == 0, (1.0, 2.5)[n // 2 % 2]
                    rows = (1, 7, 70, 130)[n % 4]
                    z, b = _logits(g, rows, E, dtype, kind), _bias(g, E, bk)
                    if n % 5 == 0:
                        say("route", E, groups, topk_groups, topk, score, dtype, kind, bk, top)
                    ids, w = gq.gq_moe_route(
                        z.to(dev), topk, score=score, bias=None if b is None else b.to(dev),
                        groups=groups, topk_groups=topk_groups, group_top=top, renormalize=renorm,
                        scale=scale)
                    torch.cuda.synchronize()
                    zn = z.float().numpy()
                    want = _select(zn, topk, score, None if b is None else b.numpy(), groups,
                                   topk_groups, top)
                    got = ids.cpu().numpy()
                    assert np.array_equal(got, want), (dtype, kind, bk, top, np.argwhere(
                        (got != want).any(axis=1))[:4].tolist())
                    _check_weights(w, zn, want, score, renorm, scale)
                    assert not w.cpu().numpy()[want < 0].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,groups,topk_groups,topk", [(128, 1, 1, 8), (256, 8, 4, 8), (60, 12, 3, 6),
                                                       (288, 8, 4, 8), (256, 4, 2, 16),
                                                       (64, 16, 5, 9), (512, 16, 4, 8),
                                                       (128, 8, 3, 8), (256, 2, 1, 16),
                                                       (200, 1, 1, 5), (48, 3, 2, 6),
                                                       (96, 2, 1, 4), (256, 16, 3, 16)])
def test_many_rows(E, groups, topk_groups, topk, dtype):
    dev = device()
    g = torch.Generator().manual_seed(E + groups)
    rows = 16384 + 5
    n = 0
    for score in ("sigmoid", "softmax"):
        for kind in ("random", "ties", "masked"):
            for bk in (None, "random", "zero"):
                top = 1 + n % 2 if groups > 1 else 1
                n += 1
                z, b = _logits(g, rows, E, dtype, kind), _bias(g, E, bk)
                say("route many", E, groups, topk, dtype, score, kind, bk, top)
                ids, w = gq.gq_moe_route(z.to(dev), topk, score=score,
                                         bias=None if b is None else b.to(dev), groups=groups,
                                         topk_groups=topk_groups, group_top=top,
                                         renormalize=n % 3 != 0)
                torch.cuda.synchronize()
                zn = z.float().numpy()
                want = _select(zn, topk, score, None if b is None else b.numpy(), groups,
                               topk_groups, top)
                assert np.array_equal(ids.cpu().numpy(), want), (score, kind, bk, top)
                _check_weights(w, zn, want, score, n % 3 != 0, 1.0)


@pytest.mark.parametrize("rows", [5, 700, 4500])
@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (60, 12)])
def test_groups_whose_choices_cancel(E, groups, rows):
    """Biases of both signs in each group, far above the scores: a group's sum is
    small where its choices' own roundings in float32 are not; and a masked-out
    group of the lowest value."""
    dev = device()
    g = np.random.default_rng(23)
    size = E // groups
    b = np.full((groups, size), -40000.0, dtype=np.float32)
    b[:, 0] = 16384.0
    b[:, size // 2] = -16384.0 + np.float32(2.0 ** -10) * g.integers(-40, 40, groups)
    b[1] = -3.4e38
    b = b.reshape(-1)
    z = (g.standard_normal((rows, E)) * 2).astype(np.float32)
    topk = min(6, 2 * size)
    for score in ("sigmoid", "softmax"):
        say("route cancelling", E, groups, rows, score)
        ids, w = gq.gq_moe_route(torch.tensor(z).to(dev), topk, score=score,
                                 bias=torch.tensor(b).to(dev), groups=groups, topk_groups=4,
                                 group_top=2)
        torch.cuda.synchronize()
        want = _select(z, topk, score, b, groups, 4, 2)
        assert np.array_equal(ids.cpu().numpy(), want), score
        _check_weights(w, z, want, score, True, 1.0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_choices_as_close_as_float64_tells(score):
    """Biases that make up for the scores' differences, so that choices agree to
    1e-8 and less and only float64 tells them apart; exact ties among them."""
    dev = device()
    g = np.random.default_rng(17)
    E, rows = 256, 4200
    z = (g.standard_normal((1, E)) * 1.5).astype(np.float32)
    z[0, 128:] = z[0, :128]                                 # pairs of equal logits
    z = np.repeat(z, rows, axis=0)
    z[1::2] += np.float32(1e-3) * g.standard_normal((rows // 2, E)).astype(np.float32)
    s = _scores(z, score)[0]
    bias = (0.75 - s).astype(np.float32)                    # every choice next to 0.75
    for groups, open_, top in ((1, 1, 1), (8, 3, 2), (8, 3, 1), (32, 9, 2)):
        say("route close", score, groups, top)
        ids, _ = gq.gq_moe_route(to_dev(z, dev), 8, score=score, bias=to_dev(bias, dev),
                                 groups=groups, topk_groups=open_, group_top=top)
        torch.cuda.synchronize()
        want = _select(z, 8, score, bias, groups, open_, top)
        assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("rows", [3, 5000])
def test_nan_and_infinity(rows):
    """A NaN is chosen first; a sigmoid's infinity is an ordinary score of one."""
    dev = device()
    z = torch.randn(rows, 64, generator=torch.Generator().manual_seed(5))
    z[0, 40] = float("nan")
    z[1, 9] = INF
    z[1, 7] = INF
    z[2, 3] = float("nan")
    z[2, 50] = INF
    b = torch.randn(64, generator=torch.Generator().manual_seed(6)) * 0.1
    say("route nan", rows)
    for bias in (None, b.to(dev)):
        for renorm in (True, False):
            ids, w = gq.gq_moe_route(z.to(dev), 4, score="sigmoid", bias=bias, groups=8,
                                     topk_groups=3, group_top=2, renormalize=renorm)
            torch.cuda.synchronize()
            want = _select(z.numpy(), 4, "sigmoid", None if bias is None else b.numpy(), 8, 3, 2)
            ids, w = ids.cpu().numpy(), w.cpu().numpy()
            assert np.array_equal(ids, want)
            assert ids[0, 0] == 40 and ids[2, 0] == 3
            if bias is None:
                assert sorted(ids[1, :2]) == [7, 9] and not np.isnan(w[1]).any()
            assert np.isnan(w[0, 0]) and np.isnan(w[0]).all() == renorm
            assert not np.isnan(w[3:]).any()
        ids, w = gq.gq_moe_route(z.to(dev), 4, bias=bias)
        torch.cuda.synchronize()
        assert np.isnan(w.cpu().numpy()[:3]).all() and not np.isnan(w.cpu().numpy()[3:]).any()
        want = _select(z.numpy(), 4, "softmax", None if bias is None else b.numpy(), 1, 1, 1)
        assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("rows", [9, 4500])
def test_agrees_with_the_softmax_topk(rows):
    """Without bias, groups and scale it is gq_moe_topk, gradient included."""
    dev = device()
    g = torch.Generator().manual_seed(rows)
    for dtype in DTYPES:
        for renorm in (True, False):
            z = _logits(g, rows, 128, dtype, "masked").to(dev)
            say("route and topk", rows, dtype, renorm)
            a, wa = gq.gq_moe_topk(z, 8, renormalize=renorm)
            b, wb = gq.gq_moe_route(z, 8, renormalize=renorm)
            dw = torch.randn(rows, 8, generator=g).to(dev)
            da = gq.gq_moe_topk_backward(dw, z, a, renormalize=renorm)
            db = gq.gq_moe_route_backward(dw, z, b, renormalize=renorm)
            torch.cuda.synchronize()
            assert torch.equal(a, b) and torch.equal(da, db)
            # two float32 evaluations of one weight
            assert ((wa - wb).abs() <= 100 * U * wa).all()


def _grad(z, ids, dw, score, renorm, scale):
    """float64 gradient slot by slot, and the magnitudes its roundings scale with."""
    z = z.astype(np.float64)
    rows, E = z.shape
    ok = (ids >= 0) & (ids < E)
    w, zs = _weights(z, np.where(ok, ids, -1), score, renorm, 1.0)
    ok &= zs > -INF
    w = np.where(ok, w, 0)
    G = np.where(ok, dw.astype(np.float64) * scale, 0)
    dot, mag = (w * G).sum(axis=1, keepdims=True), (w * np.abs(G)).sum(axis=1, keepdims=True)
    out, room = np.zeros((rows, E + 1)), np.zeros((rows, E + 1))
    at = np.where(ok, ids, E)
    r = np.arange(rows)[:, None]
    if score == "sigmoid":
        anti = np.where(ok, _scores(-np.where(ok, zs, 0), "sigmoid"), 0)
        np.add.at(out, (r, at), w * anti * (G - (dot if renorm else 0)))
        np.add.at(room, (r, at), w * anti * (np.abs(G) + (mag if renorm else 0)))
    else:
        np.add.at(out, (r, at), w * (G - (dot if renorm else 0)))
        np.add.at(room, (r, at), w * (np.abs(G) + (mag if renorm else 0)))
        if not renorm:
            p = _scores(z, "softmax")
            out[:, :E] -= p * dot
            room[:, :E] += p * mag
    return out[:, :E], room[:, :E]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("rows,E,topk", [(1, 1, 1), (7, 5, 5), (70, 60, 6), (33, 256, 8),
                                         (9, 1000, 33), (4100, 128, 8), (4096, 256, 16),
                                         (4097, 60, 6), (4100, 300, 8)])
def test_backward(rows, E, topk, score):
    dev = device()
    g = torch.Generator().manual_seed(rows + E + topk)
    for dtype in DTYPES:
        for kind in ("random", "masked", "low"):
            for renorm in (True, False):
                z = _logits(g, rows, E, dtype, kind)
                ids, _ = gq.gq_moe_route(z.to(dev), topk, score=score, renormalize=renorm)
                ids = ids.cpu()
                if E > 2 and topk > 2:                     # a repeated id, ids outside the bank
                    ids[0, 1] = ids[0, 0]
                    ids[-1, 0] = E
                    ids[-1, 2] = -7
                dw = torch.randn(rows, topk, generator=g)
                say("route backward", rows, E, topk, score, dtype, kind, renorm)
                got = gq.gq_moe_route_backward(dw.to(dev), z.to(dev), ids.to(dev), score=score,
                                               renormalize=renorm, scale=2.5)
                torch.cuda.synchronize()
                zn = z.float().numpy()
                want, room = _grad(zn, ids.numpy(), dw.numpy(), score, renorm, 2.5)
                live = zn[zn > -INF]
                far = np.abs(live).max() if live.size else 0
                # as a weight's rounding, twice (the slot's and the sum's)
                room = room * (8 * far + 200) * U
                eps = torch.finfo(dtype).eps / 2
                least = {torch.float16: 2.0 ** -25}.get(dtype, 2.0 ** -125)
                bad = np.abs(got.double().cpu().numpy() - want) > (
                    eps * (np.abs(want) + room) + room + least)
                assert not bad.any(), np.argwhere(bad)[:6].tolist()


def test_backward_against_differences():
    dev = device()
    z = torch.randn(3, 24, generator=torch.Generator().manual_seed(1)).to(dev)
    dw = torch.randn(3, 4, generator=torch.Generator().manual_seed(2)).to(dev)
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            kw = dict(score=score, renormalize=renorm, scale=1.5)
            say("route differences", score, renorm)
            ids, _ = gq.gq_moe_route(z, 4, **kw)
            grad = gq.gq_moe_route_backward(dw, z, ids, **kw)
            step = 2.0 ** -8
            for at in [(0, int(ids[0, 0])), (1, int(ids[1, 2])), (2, int(ids[2, 3])), (2, 5)]:
                side = []
                for d in (step, -step):
                    moved = z.clone()
                    moved[at] += d
                    w, _ = _weights(moved.cpu().numpy(), ids.cpu().numpy(), score, renorm, 1.5)
                    side.append((w * dw.cpu().numpy()).sum())
                # central difference: third derivatives of order one times step^2 / 6
                assert abs((side[0] - side[1]) / (2 * step) - float(grad[at])) < 2e-5


def test_strides_streams_and_graphs():
    """Rows cut out of a wider tensor; a captured call replayed on new logits and
    biases with eager calls between; another stream; buffers that are passed in."""
    dev = device()
    g = torch.Generator().manual_seed(9)
    wide = torch.randn(300, 263, generator=g).to(torch.bfloat16).to(dev)
    z, b = wide[:, 3:259], (torch.randn(256, generator=g) * 0.1).to(dev)
    dw = torch.randn(300, 8, generator=g).to(dev)
    kw = dict(score="sigmoid", scale=2.5)

    def both():
        ids, w = gq.gq_moe_route(z, 8, bias=b, groups=8, topk_groups=4, group_top=2, **kw)
        return ids, w, gq.gq_moe_route_backward(dw, z, ids, **kw)

    say("route graph")
    first = both()
    torch.cuda.synchronize()
    want = _select(z.float().cpu().numpy(), 8, "sigmoid", b.cpu().numpy(), 8, 4, 2)
    assert np.array_equal(first[0].cpu().numpy(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(4):
        wide.copy_(torch.roll(wide, i + 1, 1))
        b.neg_()
        graph.replay()
        eager = both()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, eager)), i
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = both()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(again, eager))
    ids = torch.full((300, 8), 99, dtype=torch.int32, device=dev)
    w = torch.full((300, 8), float("nan"), device=dev)
    grad = torch.full((300, 256), float("nan"), dtype=torch.bfloat16, device=dev)
    got = gq.gq_moe_route(z, 8, bias=b, groups=8, topk_groups=4, group_top=2, topk_ids=ids,
                          topk_weights=w, **kw)
    assert got[0] is ids and got[1] is w
    assert gq.gq_moe_route_backward(dw, z, ids, out=grad, **kw) is grad
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((ids, w, grad), eager))
    none = gq.gq_moe_route(z[:0], 8)
    assert none[0].shape == none[1].shape == (0, 8)
    assert gq.gq_moe_route_backward(dw[:0], z[:0], none[0]).shape == (0, 256)


def test_refusals_of_the_binding():
    dev = device()
    z = torch.zeros(4, 12, device=dev)
    for kw in (dict(topk=0), dict(topk=13), dict(topk=2, score="tanh"), dict(topk=2, groups=5),
               dict(topk=2, groups=0), dict(topk=2, groups=4, topk_groups=5),
               dict(topk=7, groups=4, topk_groups=2), dict(topk=2, groups=4, group_top=3),
               dict(topk=2, bias=torch.zeros(11, device=dev)), dict(topk=2, scale=INF),
               dict(topk=2, bias=torch.zeros(12, dtype=torch.bfloat16, device=dev)),
               dict(topk=2, topk_ids=torch.zeros(4, 3, dtype=torch.int32, device=dev))):
        with pytest.raises((ValueError, gq.GQError)):
            gq.gq_moe_route(z, **kw)
    ids = torch.zeros(4, 2, dtype=torch.int32, device=dev)
    dw = torch.zeros(4, 2, device=dev)
    for args, kw in (((dw[:3], z, ids), {}), ((dw, z, ids.long()), {}), ((dw, z[0], ids), {}),
                     ((dw, z, ids), dict(score=1)), ((dw, z, ids), dict(scale=float("nan"))),
                     ((dw, z, ids), dict(out=z[:3]))):
        with pytest.raises((ValueError, gq.GQError)):
            gq.gq_moe_route_backward(*args, **kw)


# ---- the block that norm, routing and 8-bit products make -----------------------------
def test_a_block_in_eight_bits():
    """Residual, norm, router logits, routing with groups, gate_up with the unit,
    quantisation of the result, down product with the router weights, combine:
    each step against the float64 step on the same bytes; then the single-token
    forms on its first rows."""
    dev = device()
    g = np.random.default_rng(21)
    E, H, I, M, topk = 8, 288, 320, 150, 3
    gu, dn = packed_mx_bank(g, E, 2 * I, H), packed_mx_bank(g, E, H, I)
    gud, dnd = (tuple(to_dev(t, dev) for t in b) for b in (gu, dn))
    tg = torch.Generator().manual_seed(4)
    x = torch.randn(M, H, generator=tg).to(torch.bfloat16).to(dev)
    res = torch.randn(M, H, generator=tg).to(torch.bfloat16).to(dev)
    gain = (1 + 0.1 * torch.randn(H, generator=tg)).to(torch.bfloat16).to(dev)
    router = torch.randn(E, H, generator=tg).to(torch.bfloat16).to(dev)
    bias = (torch.randn(E, generator=tg) * 0.1).to(dev)
    say("block of eight bits")
    n = gq.gq_rms_norm(x, gain, residual=res, mxfp8=True)
    logits = n.y @ router.t()
    ids, w = gq.gq_moe_route(logits, topk, score="sigmoid", bias=bias, groups=4, topk_groups=2,
                             group_top=2, scale=2.5)
    act = gq.gq_mxfp4_grouped_gemm_fp8_swiglu(n.mxfp8, *gud, gq.gq_route_sort(ids, E))
    aq = gq.gq_mxfp8_quantize(act)
    pairs = gq.gq_mxfp4_grouped_gemm_fp8(aq, *dnd, gq.gq_route_sort(ids.reshape(-1, 1), E),
                                         pair_scale=w.reshape(-1))
    y = gq.gq_moe_combine(pairs, topk)
    torch.cuda.synchronize()

    def values(q):
        codes, scales = (t.cpu().numpy() for t in q)
        v = oracle.E4M3_VALUES[codes].reshape(codes.shape[0], -1, 32)
        return np.ldexp(v, scales.astype(np.int64)[..., None] - 127).reshape(codes.shape)

    def product(xv, W, ids):
        out = np.zeros((ids.size, W(0).shape[0]))
        for e in range(E):
            at = np.nonzero(ids.reshape(-1) == e)[0]
            out[at] = xv[at // ids.shape[1]] @ W(e).astype(np.float64).T
        return out

    def check(got, ref):
        got = bf16_to_host_f32(got).astype(np.float64)
        rms = np.sqrt((ref ** 2).mean(axis=1, keepdims=True))
        assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2e-4 * rms).all()

    i = ids.cpu().numpy()
    assert np.array_equal(i, _select(logits.float().cpu().numpy(), topk, "sigmoid",
                                     bias.cpu().numpy(), 4, 2, 2))
    xv = values(n.mxfp8)
    # 8 bits hold the norm to half a step of e4m3 (2^-4) of each value, and of the
    # block's least step for small ones
    yv = n.y.double().cpu().numpy()
    top = np.repeat(np.abs(yv).reshape(M, -1, 32).max(axis=2), 32, axis=1)
    assert (np.abs(xv - yv) <= (2.0 ** -4 + 2.0 ** -7) * np.abs(yv) + 2.0 ** -17 * top).all()
    check(act, oracle.swiglu_oss(product(xv, LazyDecoded("mx", *gu), i)))
    check(pairs, product(values(aq), LazyDecoded("mx", *dn), i.reshape(-1, 1))
          * w.cpu().numpy().reshape(-1, 1))
    check(y, bf16_to_host_f32(pairs).astype(np.float64).reshape(M, topk, H).sum(axis=1))
    few = tuple(t[:4].contiguous() for t in n.mxfp8)
    one = gq.gq_mxfp4_grouped_gemv_fp8_swiglu(few, *gud, ids[:4].contiguous())
    oq = gq.gq_mxfp8_quantize(one)
    down = gq.gq_mxfp4_grouped_gemv_fp8(oq, *dnd, ids[:4].reshape(-1, 1).contiguous(),
                                        pair_scale=w[:4].reshape(-1).contiguous())
    torch.cuda.synchronize()
    check(one, oracle.swiglu_oss(product(xv[:4], LazyDecoded("mx", *gu), i[:4])))
    check(down, product(values(oq), LazyDecoded("mx", *dn), i[:4].reshape(-1, 1))
          * w[:4].cpu().numpy().reshape(-1, 1))
