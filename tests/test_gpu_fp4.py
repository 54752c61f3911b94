"""MXFP4 x MXFP4 grouped products on the GPU against the float64 product of
the decoded codes: tile edges, ragged segments, K tails, dropped pairs, the
gated unit, the single-token form, and a whole 4-bit layer of them."""

import numpy as np
import pytest
import torch

import bit_grouped_moe_amd as gq
import oracle
import workloads as wl
from tests.gpu_common import (LazyDecoded, bf16_bits, bf16_to_host_f32, device, packed_mx_bank,
                              plus_zero, say, to_dev, to_dev_bf16)

pytestmark = pytest.mark.gpu

# One rounding to bf16 (half a step, 2^-8 of the value) of a float32 sum whose
# terms are exact: K / 64 instruction results are added one after the other
# and 64 products inside each, at most K additions with 2^-24 of the sum of
# magnitudes each in the worst case; for random terms far below 2^-24 sqrt(K)
# sqrt(K) of the result, 2e-4 for K = 2880.
ROUND, SUMS = 2.0 ** -8, 2e-4


def _x(g, rows, K):
    """MXFP4 activations: oracle bytes, and their values in float64."""
    x = g.standard_normal((rows, K), dtype=np.float32)
    blocks, scales = oracle.mxfp4_pack(x)
    return (blocks, scales), oracle.mxfp4_decode(blocks, scales).astype(np.float64)


def _ref(xv, W, ids, E, N, pair_scale=None):
    ids = np.asarray(ids)
    flat = ids.reshape(-1)
    out = np.zeros((flat.size, N))
    for e in range(E):
        at = np.nonzero(flat == e)[0]
        if at.size:
            out[at] = xv[at // ids.shape[1]] @ W(e).astype(np.float64).T
    return out if pair_scale is None else out * pair_scale.reshape(-1)[:, None].astype(np.float64)


def _check(got, ref, what=""):
    got = bf16_to_host_f32(got).astype(np.float64)
    rms = np.sqrt((ref ** 2).mean(axis=1, keepdims=True))
    bad = np.abs(got - ref) > ROUND * np.abs(ref) + SUMS * rms
    assert not bad.any(), (what, np.argwhere(bad)[:8].tolist())
    assert not got[~ref.any(axis=1)].any()


def _both(x, dev):
    return tuple(to_dev(t, dev) for t in x)


@pytest.mark.parametrize("N,K", [(32, 32), (96, 64), (288, 96), (160, 256), (544, 288), (256, 512),
                                 (320, 544), (288, 1056), (544, 2048), (96, 2880)])
def test_ragged_segments(N, K):
    """Skewed routing (an expert over several tiles, others short or empty),
    widths that end inside a tile, K of one block up, dropped and
    out-of-range ids, pair scales."""
    dev = device()
    g = np.random.default_rng(N + 7 * K)
    E, M, topk = 6, 700, 2
    bank = packed_mx_bank(g, E, N, K)
    ids = wl.route_zipf(g, M, E, topk, s=2.5)
    ids[g.random(ids.shape) < 0.02] = -1
    ids[:, 1][ids[:, 1] == 4] = E
    x, xv = _x(g, M, K)
    sc = wl.router_weights(g, M, topk)
    say("fp4 ragged", N, K)
    route = gq.gq_route_sort(to_dev(ids, dev), E)
    out = gq.gq_mxfp4_grouped_gemm_fp4(_both(x, dev), *_both(bank, dev), route,
                                       pair_scale=to_dev(sc.reshape(-1), dev))
    torch.cuda.synchronize()
    _check(out, _ref(xv, LazyDecoded("mx", *bank), ids, E, N, sc))


@pytest.mark.parametrize("unit", [False, True])
@pytest.mark.parametrize("K,N", [(1056, 320), (2880, 288), (160, 64)])
def test_tile_edges(K, N, unit):
    """Segments at every count of active 32-row sub-tiles: 1 to 8, one row
    over, a one-row tail tile, an empty expert, dropped pairs."""
    dev = device()
    g = np.random.default_rng(K + 3 * N)
    sizes = [1, 32, 33, 64, 96, 97, 128, 129, 160, 161, 192, 224, 225, 256, 257, 384, 0]
    E = len(sizes)
    ids = np.concatenate([np.full(n, e, dtype=np.int32) for e, n in enumerate(sizes)]
                         + [np.full(7, -1, dtype=np.int32)])
    ids = g.permutation(ids).reshape(-1, 1)
    bank = packed_mx_bank(g, E, N, K)
    x, xv = _x(g, ids.shape[0], K)
    say("fp4 tile edges", K, N, unit)
    route = gq.gq_route_sort(to_dev(ids, dev), E)
    args = (_both(x, dev), *_both(bank, dev), route)
    ref = _ref(xv, LazyDecoded("mx", *bank), ids, E, N)
    if unit:
        out = gq.gq_mxfp4_grouped_gemm_fp4_swiglu(*args, alpha=1.1, limit=1.5)
        ref = oracle.swiglu_oss(ref, 1.1, 1.5) * (ids >= 0)
    else:
        out = gq.gq_mxfp4_grouped_gemm_fp4(*args)
    torch.cuda.synchronize()
    _check(out, ref)


@pytest.mark.parametrize("K", [32, 256, 1056])
def test_one_hot_probe_is_bit_exact(K):
    """x = e_k (code 2, scale 127): the output row is the decoded weight
    column, bit for bit, at every position of a stage."""
    dev = device()
    g = np.random.default_rng(11)
    E, N = 2, 128
    blocks, scales = packed_mx_bank(g, E, N, K)
    scales = g.integers(100, 150, scales.shape).astype(np.uint8)
    x = np.zeros((K, K), dtype=np.float32)
    x[np.arange(K), np.arange(K)] = 1.0
    xq = oracle.mxfp4_pack(x)
    ids = (np.arange(K, dtype=np.int32) % E).reshape(-1, 1)
    W = [oracle.mxfp4_decode(blocks[e], scales[e]) for e in range(E)]
    ref = np.stack([W[k % E][:, k] for k in range(K)])
    say("fp4 one-hot", K)
    xd, bank = _both(xq, dev), _both((blocks, scales), dev)
    out = gq.gq_mxfp4_grouped_gemm_fp4(xd, *bank, gq.gq_route_sort(to_dev(ids, dev), E))
    torch.cuda.synchronize()
    want = plus_zero(oracle.f32_to_bf16_rne(ref))
    assert np.array_equal(plus_zero(bf16_bits(out)), want)
    for at in range(0, min(K, 256), 32):
        one = gq.gq_mxfp4_grouped_gemv_fp4((xd[0][at:at + 32], xd[1][at:at + 32]), *bank,
                                           to_dev(ids[at:at + 32], dev))
        torch.cuda.synchronize()
        assert np.array_equal(plus_zero(bf16_bits(one)), want[at:at + 32])


@pytest.mark.parametrize("unit", [False, True])
@pytest.mark.parametrize("rows,topk,E,N,K", [(1, 4, 32, 320, 2880), (1, 1, 1, 64, 32),
                                             (8, 4, 6, 96, 256), (3, 2, 5, 160, 2080),
                                             (7, 3, 9, 544, 1056), (64, 4, 4, 32, 64),
                                             (2, 2, 2, 64, 8192)])
def test_single_token_form(rows, topk, E, N, K, unit):
    dev = device()
    g = np.random.default_rng(rows + N + K)
    bank = packed_mx_bank(g, E, N, K)
    ids = wl.route_uniform(g, rows, E, topk)
    if rows > 1:
        ids[1, 0] = -1
        ids[-1, -1] = E + 3
    x, xv = _x(g, rows, K)
    sc = g.uniform(0.5, 1.5, ids.shape).astype(np.float32)
    say("fp4 gemv", rows, topk, E, N, K, unit)
    args = (_both(x, dev), *_both(bank, dev), to_dev(ids, dev))
    ref = _ref(xv, LazyDecoded("mx", *bank), ids, E, N)
    live = ((ids >= 0) & (ids < E)).reshape(-1, 1)
    if unit:
        out = gq.gq_mxfp4_grouped_gemv_fp4_swiglu(*args)
        ref = oracle.swiglu_oss(ref) * live
    else:
        out = gq.gq_mxfp4_grouped_gemv_fp4(*args, pair_scale=to_dev(sc.reshape(-1), dev))
        ref = ref * sc.reshape(-1, 1)
    torch.cuda.synchronize()
    _check(out, ref)


def test_nan_scales_and_wide_exponents():
    """Scale byte 255 on either side: exactly the rows and columns that its
    block enters are NaN, through the unit too; scales far from 127 whose
    product is near 1."""
    dev = device()
    g = np.random.default_rng(5)
    E, M, N, K = 2, 40, 64, 288
    bank = packed_mx_bank(g, E, N, K)
    x, xv = _x(g, M, K)
    ids = (np.arange(M, dtype=np.int32) % E).reshape(-1, 1)
    up = (x[0], (x[1].astype(int) + 100).clip(0, 254).astype(np.uint8))
    down = (bank[0], (bank[1].astype(int) - 100).astype(np.uint8))
    say("fp4 wide exponents")
    route = gq.gq_route_sort(to_dev(ids, dev), E)
    a = gq.gq_mxfp4_grouped_gemm_fp4(_both(x, dev), *_both(bank, dev), route)
    b = gq.gq_mxfp4_grouped_gemm_fp4(_both(up, dev), *_both(down, dev), route)
    v = gq.gq_mxfp4_grouped_gemv_fp4(_both(up, dev), *_both(down, dev), to_dev(ids, dev))
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    _check(v, _ref(xv, LazyDecoded("mx", *bank), ids, E, N))
    x[1][3, 8] = 255                                      # token 3's last (half-filled) block
    x[1][8, 0] = 255
    bank[1][1, 10, 4] = 255                               # column 10 of expert 1
    say("fp4 nan scales")
    xd, bd = _both(x, dev), _both(bank, dev)
    want = np.zeros((M, N), dtype=bool)
    want[[3, 8]] = True
    want[1::2, 10] = True
    for out in (gq.gq_mxfp4_grouped_gemm_fp4(xd, *bd, route),
                gq.gq_mxfp4_grouped_gemv_fp4(xd, *bd, to_dev(ids, dev))):
        torch.cuda.synchronize()
        assert np.array_equal(out.float().cpu().isnan().numpy(), want)
    for out in (gq.gq_mxfp4_grouped_gemm_fp4_swiglu(xd, *bd, route),
                gq.gq_mxfp4_grouped_gemv_fp4_swiglu(xd, *bd, to_dev(ids, dev))):
        torch.cuda.synchronize()
        assert np.array_equal(out.float().cpu().isnan().numpy(), want[:, 0::2] | want[:, 1::2])


def test_a_layer_in_four_bits():
    """Routing, quantisation, gate_up with the unit, quantisation of the
    result, down product with the router weights, combine: each step against
    the float64 step on the same bytes."""
    dev = device()
    g = np.random.default_rng(21)
    E, H, I, M, topk = 8, 288, 320, 150, 3
    gu, dn = packed_mx_bank(g, E, 2 * I, H), packed_mx_bank(g, E, H, I)
    x = to_dev_bf16(wl.draw_bf16(g, (M, H)), dev)
    logits = torch.from_numpy(g.standard_normal((M, E)).astype(np.float32)).to(dev)
    logits[::7] = -float("inf")                           # tokens without an expert
    say("fp4 layer")
    ids, w = gq.gq_moe_topk(logits, topk)
    route = gq.gq_route_sort(ids, E)
    xq = gq.gq_mxfp4_quantize(x)
    act = gq.gq_mxfp4_grouped_gemm_fp4_swiglu(xq, *_both(gu, dev), route)
    aq = gq.gq_mxfp4_quantize(act)
    flat = gq.gq_route_sort(ids.reshape(-1, 1), E)
    pairs = gq.gq_mxfp4_grouped_gemm_fp4(aq, *_both(dn, dev), flat, pair_scale=w.reshape(-1))
    y = gq.gq_moe_combine(pairs, topk)
    torch.cuda.synchronize()
    i = ids.cpu().numpy()
    val = lambda q: oracle.mxfp4_decode(*[t.cpu().numpy() for t in q]).astype(np.float64)  # noqa: E731
    ref = oracle.swiglu_oss(_ref(val(xq), LazyDecoded("mx", *gu), i, E, 2 * I)) * (
        i.reshape(-1, 1) >= 0)
    _check(act, ref, "act")
    ref = _ref(val(aq), LazyDecoded("mx", *dn), i.reshape(-1, 1), E, H, w.cpu().numpy())
    _check(pairs, ref, "pairs")
    ref = bf16_to_host_f32(pairs).astype(np.float64).reshape(M, topk, H).sum(axis=1)
    _check(y, ref, "y")
    assert not y[::7].any()


def test_replayed_graph_and_other_stream():
    """Quantise, sort and product captured together; each of several replays,
    with new inputs and eager work between, equals the eager result."""
    dev = device()
    g = np.random.default_rng(31)
    E, M, N, K, topk = 5, 300, 288, 544, 2
    bank = _both(packed_mx_bank(g, E, N, K), dev)
    x = to_dev_bf16(wl.draw_bf16(g, (M, K)), dev)
    ids = to_dev(wl.route_uniform(g, M, E, topk), dev)

    def step():
        q = gq.gq_mxfp4_quantize(x)
        return gq.gq_mxfp4_grouped_gemm_fp4(q, *bank, gq.gq_route_sort(ids, E))

    say("fp4 graph")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        first = step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = step()
    assert torch.equal(first, step())
    for k in range(4):
        x.mul_(0.5 if k % 2 else -3.0)
        eager = step()
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), k


def test_binding_refuses_what_disagrees():
    dev = device()
    g = np.random.default_rng(2)
    bank = _both(packed_mx_bank(g, 3, 64, 96), dev)
    x = _both(_x(g, 5, 96)[0], dev)
    ids = torch.zeros(5, 1, dtype=torch.int32, device=dev)
    route = gq.gq_route_sort(ids, 3)
    other = _both(_x(g, 5, 128)[0], dev)
    for bad in ((other, *bank, route), ((x[0], other[1]), *bank, route),
                ((x[0].flatten(1), x[1]), *bank, route), (x, bank[0], bank[0], route),
                (x, *bank, gq.gq_route_sort(ids[:4], 3)), (x, *bank, gq.gq_route_sort(ids, 4))):
        with pytest.raises(ValueError):
            gq.gq_mxfp4_grouped_gemm_fp4(*bad)
    with pytest.raises(ValueError):
        gq.gq_mxfp4_grouped_gemv_fp4(x, *bank, ids[:4])
    with pytest.raises(ValueError):
        gq.gq_mxfp4_grouped_gemm_fp4(x, *bank, route, pair_scale=torch.ones(4, device=dev))
    empty = gq.gq_mxfp4_grouped_gemm_fp4((x[0][:0], x[1][:0]), *bank, gq.gq_route_sort(ids[:0], 3))
    assert empty.shape == (0, 64)


@pytest.mark.parametrize("unit", [False, True])
@pytest.mark.parametrize("rows,topk,E,N,K", [
    (64, 4, 4, 250, 1056), (64, 4, 4, 130, 1056),         # rows inside a wave, 8 and 4 a thread
    (64, 4, 4, 42, 2080), (64, 4, 4, 20, 2080),           # rows that meet in LDS, 8 and 4
    (16, 4, 5, 64, 8192), (16, 4, 5, 32, 8192),           # the same, one row's segments a workgroup
])
def test_single_token_form_at_every_row_count(rows, topk, E, N, K, unit):
    dev = device()
    g = np.random.default_rng(rows + 3 * N + K)
    bank = packed_mx_bank(g, E, N, K)
    ids = wl.route_uniform(g, rows, E, topk)
    ids[2, 1] = -1
    x, xv = _x(g, rows, K)
    say("fp4 gemv row counts", rows, topk, E, N, K, unit)
    args = (_both(x, dev), *_both(bank, dev), to_dev(ids, dev))
    ref = _ref(xv, LazyDecoded("mx", *bank), ids, E, N)
    if unit:
        out = gq.gq_mxfp4_grouped_gemv_fp4_swiglu(*args, alpha=1.3, limit=2.0)
        ref = oracle.swiglu_oss(ref, 1.3, 2.0) * (ids >= 0).reshape(-1, 1)
    else:
        out = gq.gq_mxfp4_grouped_gemv_fp4(*args)
    torch.cuda.synchronize()
    _check(out, ref)


@pytest.mark.parametrize("unit", [False, True])
@pytest.mark.parametrize("N,K,M", [(1056, 96, 900), (2336, 64, 300), (3328, 288, 40)])
def test_more_columns_than_a_group_of_tiles(N, K, M, unit):
    """Widths of several groups of column tiles, the last one partly filled,
    with row tiles of every kind and dropped pairs."""
    dev = device()
    g = np.random.default_rng(N + K + M)
    E, topk = 5, 2
    bank = packed_mx_bank(g, E, N, K)
    ids = wl.route_zipf(g, M, E, topk, s=2.0)
    ids[g.random(ids.shape) < 0.05] = -1
    x, xv = _x(g, M, K)
    say("fp4 column groups", N, K, M, unit)
    args = (_both(x, dev), *_both(bank, dev), gq.gq_route_sort(to_dev(ids, dev), E))
    ref = _ref(xv, LazyDecoded("mx", *bank), ids, E, N)
    shape = (M * topk, N // 2 if unit else N)
    out = torch.full(shape, float("nan"), dtype=torch.bfloat16, device=dev)
    if unit:
        gq.gq_mxfp4_grouped_gemm_fp4_swiglu(*args, out=out)
        ref = oracle.swiglu_oss(ref) * (ids >= 0).reshape(-1, 1)
    else:
        gq.gq_mxfp4_grouped_gemm_fp4(*args, out=out)
    torch.cuda.synchronize()
    _check(out, ref)
