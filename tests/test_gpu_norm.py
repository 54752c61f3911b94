"""The root-mean-square norm, its 8-bit output and its gradient on the GPU
against their definition in float64, and MXFP8 codes bit for bit."""

import numpy as np
import pytest
import torch

import bit_grouped_moe_amd as gq
import oracle
from tests.gpu_common import bf16_bits, device, say, to_dev, unpermute_split

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
TYPES = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
         (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
         (torch.float16, torch.float32)]
U = 2.0 ** -24                                  # half a float32 step
# A row's sum of squares adds at most 32 terms in a lane, 6 levels of lanes and 16
# waves: 54 roundings and one of each square; the root halves that, and the
# division, the root, its inverse and two products add 5.
NORM = (55 / 2 + 5) * U


def _half(dtype):
    """Half a step of the type relative to the value, and absolutely in its subnormals."""
    return torch.finfo(dtype).eps / 2, {torch.float16: 2.0 ** -25}.get(dtype, 2.0 ** -134)


def _inputs(rows, H, dtype, wtype, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed + 1000 * rows + H)
    x = torch.randn(rows, H + pad, generator=g) * torch.exp2(
        torch.randint(-2, 4, (1, H + pad), generator=g).float())
    r = torch.randn(rows, H + pad, generator=g)
    w = 1 + 0.3 * torch.randn(H, generator=g)
    return x.to(dtype)[:, pad:], r.to(dtype)[:, pad:], w.to(wtype)


def _sum(x, r):
    """The stored residual sum: one rounding of the float32 sum."""
    return x if r is None else (x.float() + r.float()).to(x.dtype)


def _norm(h, w, eps):
    h = h.double()
    return h / torch.sqrt((h * h).mean(dim=-1, keepdim=True) + eps) * w.double()


def _close(got, want, room, dtype, what):
    """One rounding to the type of a value that is off by at most `room`."""
    rel, least = _half(dtype)
    bad = (got.double().cpu() - want).abs() > rel * (want.abs() + room) + room + least
    assert not bad.any(), (what, bad.nonzero()[:6].tolist())


def _values_are_nearest(codes, scales, values, y):
    """Each block's scale holds its largest value without saturating and is the
    smallest that does; each code is the nearest to y (float64), all up to y's
    own error in float32."""
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy().astype(np.int64)
    y = y.numpy().reshape(-1, 32)
    X = scales.reshape(-1) - 127
    amax = np.abs(y).max(axis=1)
    room = 2 * NORM
    live = amax > 0
    assert (amax * np.exp2(-X.astype(float)) <= 448 * (1 + room))[live].all()
    assert (amax * np.exp2(1 - X.astype(float)) > 448 * (1 - room))[live & (X > -127)].all()
    v = oracle.E4M3_VALUES[codes.reshape(-1, 32)] * np.exp2(X.astype(float))[:, None]
    large = np.maximum(np.abs(v), np.abs(y)) * np.exp2(-X.astype(float))[:, None]
    e = np.maximum(np.floor(np.log2(np.maximum(large, 2.0 ** -9))), -6)
    step = np.exp2(e - 3 + X[:, None])
    bad = np.abs(v - y) > step / 2 + room * np.abs(y)
    assert not bad.any(), np.argwhere(bad)[:6].tolist()
    assert np.array_equal(values.double().cpu().numpy().reshape(-1, 32), v)


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("rows,H,pad", [(1, 1, 0), (5, 7, 3), (3, 8, 0), (130, 33, 1), (9, 511, 0),
                                        (7, 512, 8), (6, 513, 0), (3, 1024, 0), (70, 1025, 5),
                                        (4, 2048, 0), (3, 2049, 1), (1, 2880, 0), (5, 4095, 0),
                                        (3, 4097, 7), (2, 8192, 0), (2, 8193, 0), (3, 16385, 1),
                                        (2, 32768, 0)])
def test_norm(dtype, wtype, rows, H, pad):
    dev = device()
    x, r, w = _inputs(rows, H, dtype, wtype, pad)
    for res in (None, r):
        say("norm", dtype, wtype, rows, H, pad, res is not None)
        got = gq.gq_rms_norm(x.to(dev), w.to(dev), eps=1e-5,
                             residual=None if res is None else res.to(dev))
        torch.cuda.synchronize()
        h = _sum(x, res)
        assert (got.residual is None) == (res is None) and got.mxfp8 is got.values is None
        if res is not None:
            assert torch.equal(got.residual.cpu(), h)
        assert got.y.dtype == dtype and got.y.is_contiguous()
        want = _norm(h, w, 1e-5)
        _close(got.y, want, NORM * want.abs(), dtype, "y")


def test_rows_lie_at_any_stride():
    """Rows cut out of wider buffers, at odd addresses, in three dimensions."""
    dev = device()
    wide = torch.randn(6, 5, 101, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    res = torch.randn(6, 5, 203, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    w = torch.rand(96) + 0.5
    say("norm strides")
    wd, rd = wide.to(dev), res.to(dev)
    got = gq.gq_rms_norm(wd[..., 3:99], w.to(dev), residual=rd[..., 7:103], mxfp8=True, values=True)
    torch.cuda.synchronize()
    x, r = wide[..., 3:99], res[..., 7:103]
    h = _sum(x, r)
    assert torch.equal(got.residual.cpu(), h)
    want = _norm(h, w, 1e-6)
    _close(got.y, want, NORM * want.abs(), torch.bfloat16, "y")
    assert got.mxfp8[0].shape == (6, 5, 96) and got.mxfp8[1].shape == (6, 5, 3)
    _values_are_nearest(*got.mxfp8, got.values, want.reshape(30, 96))
    assert torch.equal(wd.cpu(), wide) and torch.equal(rd.cpu(), res)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H", [(1, 32), (4, 2880), (300, 96), (37, 544), (5, 2048), (3, 4128),
                                    (2, 8192), (2, 16416)])
def test_eight_bit_output(dtype, rows, H):
    dev = device()
    x, r, w = _inputs(rows, H, dtype, torch.float32, seed=7)
    x[0, :32] = 0
    r[0, :32] = 0
    say("norm mxfp8", dtype, rows, H)
    xd, rd, wd = x.to(dev), r.to(dev), w.to(dev)
    got = gq.gq_rms_norm(xd, wd, residual=rd, mxfp8=True, values=True)
    only = gq.gq_rms_norm(xd, wd, residual=rd, y=False, mxfp8=True)
    torch.cuda.synchronize()
    want = _norm(_sum(x, r), w, 1e-6)
    _values_are_nearest(*got.mxfp8, got.values, want)
    assert only.y is None and torch.equal(only.residual, got.residual)
    assert all(torch.equal(a, b) for a, b in zip(only.mxfp8, got.mxfp8))
    if dtype is torch.float32:                  # y is the unrounded result: the same bytes
        codes, scales, values = gq.gq_mxfp8_quantize(got.y, values=True)
        torch.cuda.synchronize()
        assert torch.equal(codes, got.mxfp8[0]) and torch.equal(scales, got.mxfp8[1])
        assert torch.equal(values, got.values)


def test_zero_rows_infinities_and_nan():
    """A zero row stays zero; an infinity or NaN stays in its own row."""
    dev = device()
    x = torch.randn(6, 128, generator=torch.Generator().manual_seed(3))
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 9] = float("nan")
    say("norm special rows")
    w = torch.rand(128) + 0.5
    got = gq.gq_rms_norm(x.to(dev), w.to(dev), mxfp8=True, values=True)
    torch.cuda.synchronize()
    y, scales = got.y.cpu(), got.mxfp8[1].cpu()
    assert not y[1].any() and (scales[1] == 0).all() and not got.values[1].any()
    assert torch.isnan(y[2, 5]) and not y[2, :5].any()
    assert scales[2, 0] == 255 and (scales[2, 1:] == 0).all() and not got.mxfp8[0][2, :32].any()
    assert torch.isnan(y[3]).all() and (scales[3] == 255).all() and torch.isnan(got.values[3]).all()
    for i in (0, 4, 5):
        want = _norm(x[i], w, 1e-6)
        _close(got.y[i], want, NORM * want.abs(), torch.float32, i)


def test_outputs_in_place():
    """The sum may replace the residual and y the input."""
    dev = device()
    for dtype, H in ((torch.bfloat16, 2880), (torch.float32, 1023), (torch.float16, 9000)):
        x, r, w = _inputs(19, H, dtype, torch.float32)
        xd, rd, wd = x.to(dev), r.to(dev), w.to(dev)
        say("norm in place", dtype, H)
        want = gq.gq_rms_norm(xd, wd, residual=rd)
        keep = [t.clone() for t in (want.y, want.residual)]
        got = gq.gq_rms_norm(xd, wd, residual=rd, y=xd, sum=rd)
        torch.cuda.synchronize()
        assert got.y is xd and got.residual is rd
        assert torch.equal(xd, keep[0]) and torch.equal(rd, keep[1])


def _backward(dy, h, w, dh, eps):
    """float64: gradients and the magnitudes that their roundings scale with."""
    dy, h, w = dy.double(), h.double(), w.double()
    rstd = 1 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + eps)
    n, g = h * rstd, dy * w
    mean = (g * n).mean(dim=1, keepdim=True)
    dx = rstd * (g - n * mean)
    room = rstd * ((NORM + 6 * U) * (g.abs() + (n * mean).abs())
                   + (2 * NORM + 60 * U) * n.abs() * (g * n).abs().mean(dim=1, keepdim=True))
    if dh is not None:
        dx, room = dx + dh.double(), room + 2 * U * dh.double().abs()
    return dx, room, (dy * n).sum(dim=0), (dy * n).abs().sum(dim=0)


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("rows,H,pad", [(1, 1, 0), (3, 5, 2), (1, 512, 0), (9, 300, 1),
                                        (2500, 96, 0), (601, 1025, 0), (77, 2048, 8),
                                        (33, 2880, 0), (1030, 4099, 1), (5, 8192, 0),
                                        (7, 10001, 0), (520, 32768, 0)])
def test_backward(dtype, wtype, rows, H, pad):
    dev = device()
    h, dy, w = _inputs(rows, H, dtype, wtype, pad, seed=5)
    dh = (dy.float() * 0.7).flip(0).to(dtype)
    hd, dyd, wd = h.to(dev), dy.to(dev), w.to(dev)
    for extra in (None, dh):
        say("norm backward", dtype, wtype, rows, H, pad, extra is not None)
        dx, dw = gq.gq_rms_norm_backward(dyd, hd, wd, eps=1e-5,
                                         d_residual=None if extra is None else extra.to(dev))
        torch.cuda.synchronize()
        want, room, wsum, wabs = _backward(dy, h, w, extra, 1e-5)
        _close(dx, want, room, dtype, "dx")
        # rows are added one after the other in a wave (at most rows / 512 of
        # them), then 4 waves, 8 of 512 workgroups, 4 and 16 runs
        deep = (rows + 511) // 512 + 4 + 8 + 4 + 16 + 3
        assert dw.dtype == wtype
        _close(dw, wsum, (deep * U + NORM) * wabs, wtype, "dw")
    alone, none = gq.gq_rms_norm_backward(dyd, hd, wd, eps=1e-5, d_weight=False)
    both, _ = gq.gq_rms_norm_backward(dyd, hd, wd, eps=1e-5)
    torch.cuda.synchronize()
    assert none is None and torch.equal(alone, both)


@pytest.mark.parametrize("rows", [256, 257])
@pytest.mark.parametrize("H", [513, 1024, 2049, 2880, 4096, 4097, 8192])
def test_few_and_many_rows(rows, H):
    """Widths whose rows take more waves while there are few of them, at both
    sides of the border: outputs, codes and gradients, and the first rows in a
    call of their own."""
    dev = device()
    x, r, w = _inputs(rows, H, torch.bfloat16, torch.bfloat16, 3, seed=9)
    xd, rd, wd = x.to(dev), r.to(dev), w.to(dev)
    say("norm of few and many rows", rows, H)
    q = H % 32 == 0
    got = gq.gq_rms_norm(xd, wd, residual=rd, mxfp8=q, values=q)
    dx, dw = gq.gq_rms_norm_backward(xd, got.residual, wd, d_residual=rd)
    own = gq.gq_rms_norm(xd[:3], wd, residual=rd[:3])
    torch.cuda.synchronize()
    h = _sum(x, r)
    assert torch.equal(got.residual.cpu(), h) and torch.equal(own.residual.cpu(), h[:3])
    want = _norm(h, w, 1e-6)
    _close(got.y, want, NORM * want.abs(), torch.bfloat16, "y")
    _close(own.y, want[:3], NORM * want[:3].abs(), torch.bfloat16, "own y")
    if q:
        _values_are_nearest(*got.mxfp8, got.values, want)
    wx, room, ws, wabs = _backward(x, h, w, r, 1e-6)
    _close(dx, wx, room, torch.bfloat16, "dx")
    deep = 1 + 4 + 8 + 4 + 16 + 3
    _close(dw, ws, (deep * U + NORM) * wabs, torch.bfloat16, "dw")


def test_backward_against_differences():
    """The gradient of a random linear function of y and h, against central
    differences of the forward kernel in float32."""
    dev = device()
    rows, H = 3, 40
    x, r, w = _inputs(rows, H, torch.float32, torch.float32, seed=11)
    g = torch.Generator().manual_seed(12)
    cy, ch = torch.randn(rows, H, generator=g), torch.randn(rows, H, generator=g)
    xd, rd, wd = x.to(dev), r.to(dev), w.to(dev)

    def f(x, w):
        n = gq.gq_rms_norm(x, w, residual=rd)
        return float((n.y.double().cpu() * cy).sum() + (n.residual.double().cpu() * ch).sum())

    say("norm differences")
    h = gq.gq_rms_norm(xd, wd, residual=rd).residual
    dx, dw = gq.gq_rms_norm_backward(cy.to(dev), h, wd, d_residual=ch.to(dev))
    step = 2.0 ** -6
    # a difference is off by the third derivative's step^2 / 6 (of order one over
    # the row's scale squared) and by float32 values' roundings over the step
    for at in [(0, 0), (1, 17), (2, 39)]:
        a, b = xd.clone(), xd.clone()
        a[at] += step
        b[at] -= step
        assert abs((f(a, wd) - f(b, wd)) / (2 * step) - float(dx[at])) < 5e-3
    for i in (0, 21, 39):
        a, b = wd.clone(), wd.clone()
        a[i] += step
        b[i] -= step
        assert abs((f(xd, a) - f(xd, b)) / (2 * step) - float(dw[i])) < 5e-3


def test_backward_is_reproducible_and_writes_in_place():
    dev = device()
    h, dy, w = _inputs(3001, 2048, torch.bfloat16, torch.bfloat16)
    hd, dyd, wd = h.to(dev), dy.to(dev), w.to(dev)
    dh = dyd.flip(0).contiguous()
    say("norm backward twice")
    dx, dw = gq.gq_rms_norm_backward(dyd, hd, wd, d_residual=dh)
    space = torch.full((gq.gq_rms_norm_backward_workspace(3001, 2048),), 255, dtype=torch.uint8,
                       device=dev)                       # NaN wherever it is read unwritten
    for into in ("d_y", "h", "d_residual"):
        a, b, c = dyd.clone(), hd.clone(), dh.clone()
        out = {"d_y": a, "h": b, "d_residual": c}[into]
        got = gq.gq_rms_norm_backward(a, b, wd, d_residual=c, d_x=out, workspace=space)
        torch.cuda.synchronize()
        assert got[0] is out and torch.equal(out, dx) and torch.equal(got[1], dw), into


def test_no_rows():
    dev = device()
    for dtype in DTYPES:
        x = torch.zeros(0, 64, dtype=dtype, device=dev)
        w = torch.ones(64, dtype=dtype, device=dev)
        say("norm no rows", dtype)
        got = gq.gq_rms_norm(x, w, residual=x, mxfp8=True, values=True)
        assert got.y.shape == got.residual.shape == (0, 64) and got.mxfp8[1].shape == (0, 2)
        dw = torch.full((64,), 7.0, dtype=dtype, device=dev)
        dx, got = gq.gq_rms_norm_backward(x, x, w, d_weight=dw)
        torch.cuda.synchronize()
        assert dx.shape == (0, 64) and got is dw and not dw.any()


def test_rows_past_32_bits():
    """Offsets past 2^31 elements: the last rows of a long tensor."""
    dev = device()
    rows, H = (1 << 31) // 2048 + 3, 2048
    x = torch.empty(rows, H, dtype=torch.bfloat16, device=dev)
    x[-4:] = torch.randn(4, H, generator=torch.Generator().manual_seed(4)).to(x)
    x[:-4] = 0
    w = torch.ones(H, device=dev)
    say("norm long")
    got = gq.gq_rms_norm(x, w, residual=x, y=True, mxfp8=True)
    few = gq.gq_rms_norm(x[-4:], w, residual=x[-4:], y=True, mxfp8=True)
    torch.cuda.synchronize()
    assert torch.equal(got.y[-4:], few.y) and torch.equal(got.residual[-4:], few.residual)
    assert torch.equal(got.mxfp8[0][-4:], few.mxfp8[0])
    assert torch.equal(got.mxfp8[1][-4:], few.mxfp8[1])
    assert not got.y[:8].any() and not got.y[-8:-4].any()
    dx, dw = gq.gq_rms_norm_backward(x, x, w)
    fx, fw = gq.gq_rms_norm_backward(x[-4:], x[-4:], w)
    torch.cuda.synchronize()
    assert torch.equal(dx[-4:], fx)
    assert torch.allclose(dw, fw, rtol=1e-5, atol=1e-6)      # other workgroups, four rows


def test_captured_and_on_a_stream():
    """Forward and backward replayed from a graph on new inputs, eager calls
    between the replays; then on a stream that is not torch's default."""
    dev = device()
    x, r, w = _inputs(300, 1056, torch.bfloat16, torch.float32, seed=21)
    sx, sr, wd = x.to(dev), r.to(dev), w.to(dev)

    def both():
        n = gq.gq_rms_norm(sx, wd, residual=sr, mxfp8=True, values=True)
        return (*n[:2], *n.mxfp8, n.values, *gq.gq_rms_norm_backward(n.y, n.residual, wd,
                                                                      d_residual=sr))

    say("norm graph")
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(4):
        sx.copy_(torch.roll(x, i, 0).to(dev) * (i + 1))
        graph.replay()
        eager = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), i
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = both()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, eager))


# ---- MXFP8 quantisation -----------------------------------------------------------
def _expect(x):
    """Oracle codes, scales and bf16 value bits of a tensor [rows, K]."""
    w = x.detach().double().cpu().numpy()
    blk = w.reshape(w.shape[0], -1, 32)
    bad = ~np.isfinite(blk).all(-1)
    blk = np.where(bad[..., None], 0, blk)
    X = oracle.block_scale_exponent(np.abs(blk).max(axis=-1))
    codes = oracle.e4m3_rne(np.ldexp(blk, -X[..., None]))
    with np.errstate(over="ignore"):            # the largest float32 values round up to 2^128
        values = np.ldexp(oracle.E4M3_VALUES[codes], X[..., None]).astype(np.float32)
    codes[bad] = 0
    scales = np.where(bad, 255, X + 127).astype(np.uint8)
    return (codes.reshape(w.shape), scales,
            oracle.f32_to_bf16_rne(values.reshape(w.shape)), np.repeat(bad, 32, axis=1))


def _check_bytes(x, got):
    codes, scales, values = got
    torch.cuda.synchronize()
    ec, es, ev, bad = _expect(x.reshape(-1, x.shape[-1]))
    assert np.array_equal(scales.cpu().numpy().reshape(es.shape), es)
    assert np.array_equal(codes.cpu().numpy().reshape(ec.shape), ec)
    gv = bf16_bits(values).reshape(ev.shape)
    assert np.array_equal((gv & 0x7FFF) > 0x7F80, bad)
    assert np.array_equal(gv[~bad], ev[~bad])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,K,pad", [(1, 32, 0), (3, 96, 0), (7, 2880, 0), (5, 64, 3),
                                        (300, 2048, 8), (2, 8192 + 32, 1), (513, 32, 7)])
def test_codes_equal_the_oracle(dtype, rows, K, pad):
    dev = device()
    g = torch.Generator().manual_seed(rows * 7 + K + pad)
    x = torch.randn(rows, K + pad + 1, generator=g) * torch.exp2(
        torch.randint(-6, 6, (rows, 1), generator=g).float())
    x = x.to(dtype).to(dev)[:, 1:1 + K]        # starts one element into the row
    say("mxfp8", dtype, rows, K, pad)
    _check_bytes(x, gq.gq_mxfp8_quantize(x, values=True))
    y = x.contiguous()
    _check_bytes(y, gq.gq_mxfp8_quantize(y, values=True))


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_code_and_border(dtype):
    """All e4m3 values, the midpoints between them and their neighbours, both
    signs, at several exponents; a block maximum around 448 times a power of two."""
    dev = device()
    mags = oracle.E4M3_VALUES[:0x7F]
    mid = (mags[1:] + mags[:-1]) / 2
    near = np.concatenate([mags, mid, mid * (1 + 2.0 ** -7), mid * (1 - 2.0 ** -7)])
    near = near[near <= 448]
    rows = []
    for e in (-14, -9, 0, 5):
        for sign in (1, -1):
            for at in range(0, len(near), 30):
                row = np.zeros(32)
                part = near[at:at + 30]
                row[:len(part)] = sign * part
                row[31] = 448.0                # fixes the block's exponent
                row[30] = -0.0
                rows.append(row * 2.0 ** e)
    for top in (446.0, 448.0, 450.0, 511.0, 512.0):
        rows.append(np.full(32, top))
    x = torch.tensor(np.array(rows), dtype=torch.float32).to(dtype).to(dev)
    say("mxfp8 borders", dtype)
    _check_bytes(x, gq.gq_mxfp8_quantize(x, values=True))


def test_tiny_huge_and_special_values():
    dev = device()
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(10, 64)
    x[0, :] = -0.0
    x[1, :3] = torch.tensor([1e-45, -3e-45, 1e-40])      # float32 subnormals
    x[2, :4] = torch.tensor([2.0 ** -126, 2.0 ** -125, -(2.0 ** -127), 2.0 ** -149])
    x[3, :3] = torch.tensor([3.4028234e38, -3e38, 1.0])
    x[4, 5] = inf
    x[5, 40] = -inf
    x[6, 31] = nan
    x[7, :] = torch.linspace(-1, 1, 64)
    x[7, 32] = nan
    x[8, :2] = torch.tensor([2.0 ** -118, 2.0 ** -130])
    x[9, :2] = torch.tensor([447 * 2.0 ** -127, 2.0 ** -134])
    say("mxfp8 special blocks")
    for t in (x, x.to(torch.bfloat16)):
        d = t.to(dev)
        _check_bytes(d, gq.gq_mxfp8_quantize(d, values=True))


def test_codes_are_the_splits_first_term():
    dev = device()
    x = torch.randn(37, 2880, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).to(dev)
    say("mxfp8 and the split")
    codes, scales = gq.gq_mxfp8_quantize(x)
    xq = gq.gq_act_split_e4m3(x)
    torch.cuda.synchronize()
    hi, _, s_hi, _ = unpermute_split(xq[0].cpu().numpy(), xq[1].cpu().numpy(), 2880)
    assert np.array_equal(codes.cpu().numpy(), hi) and np.array_equal(scales.cpu().numpy(), s_hi)


def test_values_in_place_and_requantised():
    dev = device()
    x = torch.randn(64, 2880, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).to(dev)
    say("mxfp8 values")
    codes, scales, values = gq.gq_mxfp8_quantize(x, values=True)
    again = gq.gq_mxfp8_quantize(values, values=True)
    inplace = gq.gq_mxfp8_quantize(x, values=x)
    torch.cuda.synchronize()
    assert inplace[2] is x and torch.equal(x, values)
    # a maximum just above 448 2^X takes the next exponent and may round to 448 2^X
    # there, which quantised again has the smaller exponent: other bytes, the same
    # values (of the smaller exponent's steps, every one of the larger's is one)
    assert torch.equal(again[2], values)
    decoded = codes.view(torch.float8_e4m3fn).float().unflatten(1, (-1, 32))
    decoded = torch.ldexp(decoded, scales.int().unsqueeze(2) - 127).flatten(1)
    assert torch.equal(decoded, values.float())
