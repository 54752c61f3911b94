"""MXFP4 quantisation on the GPU, bit for bit against the oracle's packer:
codes, scale bytes and the values they stand for."""

import numpy as np
import pytest
import torch

import bit_grouped_moe_amd as gq
import oracle
from tests.gpu_common import bf16_bits, device, say

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def _expect(x):
    """Oracle bytes and bf16 value bits of a device tensor [rows, K]; blocks
    with an infinity or NaN: scale 255, codes 0."""
    w = x.detach().float().cpu().numpy()
    blk = w.reshape(w.shape[0], -1, 32)
    bad = ~np.isfinite(blk).all(-1)
    blocks, scales = oracle.mxfp4_pack(np.where(bad[..., None], 0, blk).reshape(w.shape))
    blocks[bad] = 0
    scales[bad] = 255
    values = oracle.f32_to_bf16_rne(oracle.mxfp4_decode(blocks, scales))
    return blocks, scales, values


def _check(x, got):
    blocks, scales, values = got
    torch.cuda.synchronize()
    eb, es, ev = _expect(x.reshape(-1, x.shape[-1]))
    assert np.array_equal(scales.cpu().numpy().reshape(es.shape), es)
    assert np.array_equal(blocks.cpu().numpy().reshape(eb.shape), eb)
    gv = bf16_bits(values).reshape(ev.shape)
    nan = (gv & 0x7FFF) > 0x7F80
    assert np.array_equal(nan, np.repeat(es == 255, 32, axis=1))
    assert np.array_equal(gv[~nan], ev[~nan])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,K,pad", [(1, 32, 0), (3, 96, 0), (7, 2880, 0), (5, 64, 3),
                                        (300, 2048, 8), (2, 8192 + 32, 1), (513, 32, 7)])
def test_bytes_equal_the_oracle(dtype, rows, K, pad):
    dev = device()
    g = torch.Generator().manual_seed(rows * 7 + K + pad)
    x = torch.randn(rows, K + pad + 1, generator=g) * torch.exp2(
        torch.randint(-6, 6, (rows, 1), generator=g).float())
    x = x.to(dtype).to(dev)[:, 1:1 + K]        # starts one element into the row
    say("quantize", dtype, rows, K, pad)
    _check(x, gq.gq_mxfp4_quantize(x, values=True))
    y = x.contiguous()
    _check(y, gq.gq_mxfp4_quantize(y, values=True))


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_border_of_the_format(dtype):
    """All e2m1 values, all midpoints between them and their neighbours one
    step away, both signs, at several block exponents; a block maximum just
    under and at a power of two; saturation between 6 and 8."""
    dev = device()
    mags = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.5])
    near = np.concatenate([mags, mags * (1 + 2.0 ** -7), mags * (1 - 2.0 ** -7)])
    near = near[near < 8]
    rows = []
    for e in (-14, -9, 0, 5, 11):
        for sign in (1, -1):
            for at in range(0, len(near), 30):
                row = np.zeros(32)
                part = near[at:at + 30]
                row[:len(part)] = sign * part
                row[31] = 4.0                  # fixes the block's exponent
                row[30] = -0.0
                rows.append(row * 2.0 ** e)
    rows.append(np.full(32, 7.9921875))
    rows.append(np.full(32, 3.9921875))
    x = torch.tensor(np.array(rows), dtype=torch.float32).to(dtype).to(dev)
    say("quantize borders", dtype)
    _check(x, gq.gq_mxfp4_quantize(x, values=True))


def test_tiny_huge_and_special_blocks():
    dev = device()
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(9, 64)
    x[0, :] = -0.0                                       # a zero block keeps its signs
    x[1, :3] = torch.tensor([1e-45, -3e-45, 1e-40])      # float32 subnormals
    x[2, :4] = torch.tensor([2.0 ** -126, 2.0 ** -125, -(2.0 ** -127), 2.0 ** -149])
    x[3, :3] = torch.tensor([3.4028234e38, -3e38, 1.0])
    x[4, 5] = inf
    x[5, 40] = -inf
    x[6, 31] = nan
    x[7, :] = torch.linspace(-1, 1, 64)
    x[7, 32] = nan
    x[8, :2] = torch.tensor([2.0 ** -124, 2.0 ** -130])
    say("quantize special blocks")
    for t in (x, x.to(torch.bfloat16)):
        d = t.to(dev)
        _check(d, gq.gq_mxfp4_quantize(d, values=True))


def test_requantising_decoded_values_reproduces_the_bytes():
    dev = device()
    x = torch.randn(64, 2880, generator=torch.Generator().manual_seed(3)).to(dev)
    say("quantize twice")
    blocks, scales, values = gq.gq_mxfp4_quantize(x, values=True)
    again = gq.gq_mxfp4_quantize(values)
    f32, _ = gq.gq_mxfp4_decode(blocks, scales)
    third = gq.gq_mxfp4_quantize(f32)
    torch.cuda.synchronize()
    for b, s in (again, third):
        assert torch.equal(b, blocks) and torch.equal(s, scales)
    assert torch.equal(f32, values.float())


def test_values_in_place():
    """The values may replace bf16 inputs."""
    dev = device()
    x = torch.randn(37, 2880, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(dev)
    say("quantize in place")
    ref = gq.gq_mxfp4_quantize(x, values=True)
    got = gq.gq_mxfp4_quantize(x, values=x)
    torch.cuda.synchronize()
    assert got[2] is x
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_leading_dimensions_given_buffers_and_untouched_neighbours():
    dev = device()
    x = torch.randn(3, 5, 96, generator=torch.Generator().manual_seed(5)).to(dev)
    pool = torch.full((3 * 5 * 48 + 64,), 0xA5, dtype=torch.uint8, device=dev)
    spool = torch.full((3 * 5 * 3 + 8,), 0xA5, dtype=torch.uint8, device=dev)
    blocks = pool[16:16 + 720].view(3, 5, 3, 16)
    scales = spool[3:3 + 45].view(3, 5, 3)
    say("quantize into given buffers")
    b, s, v = gq.gq_mxfp4_quantize(x, values=True, blocks=blocks, scales=scales)
    assert b is blocks and s is scales and v.shape == x.shape
    _check(x, (b, s, v))
    assert (pool[:16] == 0xA5).all() and (pool[736:] == 0xA5).all()
    assert (spool[:3] == 0xA5).all() and (spool[48:] == 0xA5).all()
    e = gq.gq_mxfp4_quantize(x[:0])
    assert e[0].shape == (0, 5, 3, 16) and e[1].shape == (0, 5, 3)
    for kw in (dict(blocks=blocks[:2]), dict(scales=scales.float()), dict(values=v.float())):
        with pytest.raises(ValueError):
            gq.gq_mxfp4_quantize(x, **kw)
    with pytest.raises(gq.GQError):
        gq.gq_mxfp4_quantize(x[..., :40])              # width not a multiple of 32
    with pytest.raises(gq.GQError):
        gq.gq_mxfp4_quantize(x[0, :1].expand(4, 96))   # rows on top of each other


def test_offsets_past_32_bits():
    """Rows whose values, codes and outputs lie past 2^32 bytes."""
    dev = device()
    K = 1 << 20
    rows = 2100                                         # 2.2e9 values, 4.4 GB of bf16
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=dev)
    tail = torch.randn(2, K, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).to(dev)
    x[-2:] = tail
    say("quantize past 32 bits")
    blocks, scales, values = gq.gq_mxfp4_quantize(x, values=True)
    torch.cuda.synchronize()
    _check(tail, (blocks[-2:], scales[-2:], values[-2:]))
    assert int(scales[0, 0]) == 0 and not blocks[0].any()


def test_more_rows_than_a_launch_takes():
    """2^35 contiguous values, whose groups of eight pass the threads of a
    launch: the same bytes as the last rows and some in the middle have by
    themselves, and every block written.  Inputs and codes pass 2^32 bytes."""
    dev = device()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    rows = (1 << 30) + 5
    say("quantize many launches", rows)
    x = torch.zeros(rows, 32, dtype=torch.bfloat16, device=dev)
    at = [slice(0, 100), slice((1 << 29) - 50, (1 << 29) + 50), slice(rows - 100, rows)]
    g = torch.Generator().manual_seed(10)
    for s in at:
        x[s] = torch.randn(100, 32, generator=g).to(torch.bfloat16).to(dev)
    blocks = torch.empty(rows, 1, 16, dtype=torch.uint8, device=dev)
    blocks[rows // 3].fill_(0xA5)
    scales = torch.full((rows, 1), 0xA5, dtype=torch.uint8, device=dev)
    gq.gq_mxfp4_quantize(x, blocks=blocks, scales=scales)
    torch.cuda.synchronize()
    assert int(scales.max()) < 0xA5 and not blocks[rows // 3].any()
    for s in at:
        one = x[s].clone()
        b, c, v = gq.gq_mxfp4_quantize(one, values=True)
        torch.cuda.synchronize()
        assert torch.equal(b, blocks[s]) and torch.equal(c, scales[s])
        _check(one, (b, c, v))


def test_strided_rows_past_32_bits():
    """Rows of a wider buffer, so that a row's own offset counts: values, codes
    and bf16 values past 2^32 bytes."""
    dev = device()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    rows, K, pad = (1 << 18) + 3, 1 << 15, 40
    say("quantize strided past 32 bits", rows, K)
    room = torch.zeros(rows, K + pad, dtype=torch.bfloat16, device=dev)
    x = room[:, 8:8 + K]
    at = [slice(0, 2), slice((1 << 17) - 1, (1 << 17) + 1), slice(rows - 2, rows)]
    g = torch.Generator().manual_seed(11)
    for s in at:
        x[s] = torch.randn(2, K, generator=g).to(torch.bfloat16).to(dev)
    blocks, scales, values = gq.gq_mxfp4_quantize(x, values=True)
    torch.cuda.synchronize()
    for s in at:
        _check(x[s].contiguous(), (blocks[s], scales[s], values[s]))
    for r in (2, (1 << 17) + 1, rows - 3):
        assert not blocks[r].any() and not scales[r].any() and not values[r].any()


def test_one_row_of_more_than_32_bits():
    """A flat tensor whose length does not fit 32 bits: the bytes of its parts."""
    dev = device()
    n = (1 << 32) + 96                                   # the low half would be three blocks
    say("quantize one long row", n)
    x = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    at = [slice(0, 128), slice((1 << 31) - 64, (1 << 31) + 64), slice(n - 128, n)]
    g = torch.Generator().manual_seed(12)
    for s in at:
        x[s] = torch.randn(128, generator=g).to(torch.bfloat16).to(dev)
    blocks, scales = gq.gq_mxfp4_quantize(x)
    assert blocks.shape == (n // 32, 16) and scales.shape == (n // 32,)
    for s in at:
        b = slice(s.start // 32, s.stop // 32)
        one = x[s].clone()
        _, _, v = gq.gq_mxfp4_quantize(one, values=True)
        torch.cuda.synchronize()
        _check(one, (blocks[b], scales[b], v))
    for bad in (x[:n - 1], torch.as_strided(x, (2, 1 << 31), ((1 << 31) + 32, 1))):
        with pytest.raises(gq.GQError):                  # not whole blocks; rows with a gap
            gq.gq_mxfp4_quantize(bad)
