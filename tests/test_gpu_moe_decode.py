"""The whole decode layer (router, selection, experts, combine) on the GPU
against its formula in float64."""

import numpy as np
import pytest
import torch

import bit_grouped_moe_amd as gq
import oracle
import workloads as wl
from tests.gpu_common import (LazyDecoded, bf16_to_host_f32, device, packed_mx_bank,
                              packed_nf4_bank, say, to_dev, to_dev_bf16)

pytestmark = pytest.mark.gpu

# Output bf16: half a step is 2^-8 of the value.  The float32 sums before it:
# at most 40 additions follow one another in a dot product (32 in a lane, the
# rest a tree), so its error is below 40 2^-24 times the sum of magnitudes,
# about 40 times the result's size for 4096 random terms: 1e-4 for each of the
# two products.
ROUND, SUMS = 2.0 ** -8, 2e-4


class Case:
    """A layer's weights on host and device."""

    def __init__(self, fmt, E, H, I, topk, bias=False, renorm=True, seed=0, alpha=1.702, limit=7.0):
        g = np.random.default_rng([seed, E, H, I, topk])
        self.fmt, self.E, self.H, self.I, self.topk, self.renorm = fmt, E, H, I, topk, renorm
        self.alpha, self.limit = alpha, limit
        pack = packed_nf4_bank if fmt == "nf4" else packed_mx_bank
        self.gu, self.dn = pack(g, E, 2 * I, H), pack(g, E, H, I)
        self.router = wl.draw_bf16(g, (E, H), std=0.1)
        self.bias = [wl.draw_bf16(g, s, std=0.5) if bias else None
                     for s in ((E,), (E, 2 * I), (E, H))]
        self.g = g

    def layer(self, dev):
        b = [None if v is None else to_dev_bf16(v, dev) for v in self.bias]
        return gq.gq_moe_layer(to_dev_bf16(self.router, dev),
                               tuple(to_dev(t, dev) for t in self.gu),
                               tuple(to_dev(t, dev) for t in self.dn), self.topk,
                               router_bias=b[0], gate_up_bias=b[1], down_bias=b[2],
                               renormalize=self.renorm, alpha=self.alpha, limit=self.limit)

    def reference(self, x_bits):
        """float64 [rows, H], and the smallest gap at the border of a selection."""
        f = lambda b: oracle.bf16_to_f32(b).astype(np.float64)   # noqa: E731
        x = f(x_bits)
        z = x @ f(self.router).T
        if self.bias[0] is not None:
            z = z + f(self.bias[0])
        fmt = "nf4" if self.fmt == "nf4" else "mx"
        Wg, Wd = LazyDecoded(fmt, *self.gu), LazyDecoded(fmt, *self.dn)
        y = np.zeros((x.shape[0], self.H))
        gap = np.inf
        for t in range(x.shape[0]):
            order = np.argsort(-z[t], kind="stable")
            chosen = [e for e in order[:self.topk] if z[t, e] > -np.inf]
            top = z[t, order]
            if len(order) > self.topk and np.isfinite(top[self.topk]):
                gap = min(gap, top[self.topk - 1] - top[self.topk])
            if not chosen:
                continue
            pool = z[t, chosen] if self.renorm else z[t][z[t] > -np.inf]
            norm = np.exp(pool - top[0]).sum()
            for e in chosen:
                h = Wg(e).astype(np.float64) @ x[t]
                if self.bias[1] is not None:
                    h = h + f(self.bias[1])[e]
                if self.fmt == "nf4":
                    a = oracle.swiglu(h[None])[0]
                else:
                    a = oracle.swiglu_oss(h[None], self.alpha, self.limit)[0]
                o = Wd(e).astype(np.float64) @ a
                if self.bias[2] is not None:
                    o = o + f(self.bias[2])[e]
                y[t] += np.exp(z[t, e] - top[0]) / norm * o
        return y, gap

    def check(self, got, x_bits):
        ref, gap = self.reference(x_bits)
        assert gap > 1e-4, "two experts too close for a float32 selection: another seed"
        got = bf16_to_host_f32(got).astype(np.float64)
        for t in range(ref.shape[0]):
            rms = np.sqrt((ref[t] ** 2).mean())
            assert (np.abs(got[t] - ref[t]) <= ROUND * np.abs(ref[t]) + SUMS * rms).all(), t


def _x(case, rows, std=1.0):
    return wl.draw_bf16(case.g, (rows, case.H), std=std)


@pytest.mark.parametrize("fmt,E,H,I,topk,rows,bias,renorm", [
    ("nf4", 4, 256, 128, 2, 1, False, True),
    ("nf4", 4, 256, 128, 2, 8, True, False),
    ("nf4", 1, 64, 64, 1, 1, True, True),
    ("nf4", 9, 192, 320, 9, 7, False, False),
    ("nf4", 130, 64, 64, 8, 8, True, True),
    ("nf4", 5, 2048, 768, 3, 5, False, True),
    ("nf4", 3, 2112, 64, 2, 3, True, True),
    ("nf4", 3, 128, 2112, 2, 8, True, True),
    ("nf4", 20, 64, 4096, 8, 8, False, True),
    ("nf4", 2, 4160, 192, 2, 2, False, False),
    ("nf4", 2, 8192, 64, 1, 2, False, True),
    ("mxfp4", 4, 256, 128, 2, 1, False, True),
    ("mxfp4", 4, 96, 160, 4, 8, True, False),
    ("mxfp4", 1, 32, 32, 1, 1, True, True),
    ("mxfp4", 300, 64, 32, 8, 8, True, True),
    ("mxfp4", 4, 2880, 2880, 4, 2, True, True),
    ("mxfp4", 3, 2080, 96, 2, 3, False, True),
    ("mxfp4", 6, 544, 4096, 6, 8, True, False),
    ("mxfp4", 2, 8192, 96, 2, 1, True, True),
    ("mxfp4", 70, 32, 32, 64, 1, True, True),          # as many slots as the wave has lanes
    ("mxfp4", 500, 64, 64, 64, 1, False, False),
    ("nf4", 66, 64, 64, 32, 2, True, True),
    ("nf4", 8, 64, 4096, 8, 8, True, True),
    ("mxfp4", 5, 96, 2080, 1, 8, False, True),
])
def test_layer(fmt, E, H, I, topk, rows, bias, renorm):
    dev = device()
    c = Case(fmt, E, H, I, topk, bias, renorm)
    x = _x(c, rows)
    say("moe decode", fmt, E, H, I, topk, rows, bias, renorm)
    layer = c.layer(dev)
    y = gq.gq_moe_decode(layer, to_dev_bf16(x, dev))
    torch.cuda.synchronize()
    c.check(y, x)
    assert torch.equal(y, gq.gq_moe_decode(layer, to_dev_bf16(x, dev)))


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_same_token_many_times_and_single_rows(fmt):
    """All tokens choose the same experts; each row equals the row alone, bit
    for bit; rows of a wider buffer."""
    dev = device()
    c = Case(fmt, 12, 576, 192, 5, bias=True)
    x = _x(c, 8)
    x[3:] = x[3]
    say("moe decode same token", fmt)
    layer = c.layer(dev)
    wide = torch.zeros(8, 640, dtype=torch.bfloat16, device=dev)
    wide[:, 16:592] = to_dev_bf16(x, dev)
    y = gq.gq_moe_decode(layer, wide[:, 16:592])
    torch.cuda.synchronize()
    c.check(y, x)
    for t in (0, 3, 7):
        assert torch.equal(gq.gq_moe_decode(layer, wide[t:t + 1, 16:592])[0], y[t])


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_masked_experts_and_empty_rows(fmt):
    """A router bias of -inf masks an expert: slots without one add nothing,
    and a layer with every expert masked returns zeros."""
    dev = device()
    c = Case(fmt, 6, 128, 64, 4, bias=True)
    x = _x(c, 3)
    c.bias[0][[0, 2, 3, 5]] = 0xFF80                     # -inf
    say("moe decode masked", fmt)
    y = gq.gq_moe_decode(c.layer(dev), to_dev_bf16(x, dev))
    torch.cuda.synchronize()
    c.check(y, x)
    c.bias[0][:] = 0xFF80
    y = gq.gq_moe_decode(c.layer(dev), to_dev_bf16(x, dev))
    torch.cuda.synchronize()
    assert not y.any()


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_nan_token_stays_its_own(fmt):
    dev = device()
    c = Case(fmt, 8, 256, 128, 3)
    x = _x(c, 4)
    say("moe decode nan", fmt)
    layer = c.layer(dev)
    clean = gq.gq_moe_decode(layer, to_dev_bf16(x, dev))
    x[1, 200] = 0x7FC0
    y = gq.gq_moe_decode(layer, to_dev_bf16(x, dev))
    torch.cuda.synchronize()
    assert y[1].isnan().all()
    assert torch.equal(y[[0, 2, 3]], clean[[0, 2, 3]])


def test_unit_parameters():
    dev = device()
    c = Case("mxfp4", 5, 128, 96, 2, bias=True, alpha=0.75, limit=0.5)
    x = _x(c, 4, std=4.0)
    say("moe decode unit parameters")
    y = gq.gq_moe_decode(c.layer(dev), to_dev_bf16(x, dev))
    torch.cuda.synchronize()
    c.check(y, x)


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_against_the_separate_operators(fmt):
    """The layer against router product, gq_moe_topk, the decode GEMVs and
    their combine: the same up to those steps' bf16 rounding of the gated
    product (half a step, averaged over I terms) and of the output."""
    dev = device()
    c = Case(fmt, 16, 512, 256, 4)
    x = to_dev_bf16(_x(c, 5), dev)
    say("moe decode against separate operators", fmt)
    layer = c.layer(dev)
    y = gq.gq_moe_decode(layer, x)
    z = x.float() @ to_dev_bf16(c.router, dev).float().t()
    ids, w = gq.gq_moe_topk(z, 4)
    gu, dn = [[to_dev(t, dev) for t in b] for b in (c.gu, c.dn)]
    if fmt == "nf4":
        act = gq.gq_nf4_grouped_gemv_swiglu(x, *gu, ids)
        ref = gq.gq_nf4_grouped_gemv_down_combine(act, *dn, ids, w)
    else:
        act = gq.gq_mxfp4_grouped_gemv_swiglu(x, *gu, ids)
        ref = gq.gq_mxfp4_grouped_gemv_down_combine(act, *dn, ids, w)
    torch.cuda.synchronize()
    d, r = (y.float() - ref.float()).norm(dim=1), ref.float().norm(dim=1)
    assert (d <= 3 * ROUND * r).all()                    # three roundings, each at most one


def test_workspace_and_output_given():
    """The workspace needs no clearing, nothing is written past its size or
    the output's, and one that is too small is refused."""
    dev = device()
    c = Case("nf4", 10, 320, 128, 3)
    x = to_dev_bf16(_x(c, 6), dev)
    say("moe decode workspace")
    layer = c.layer(dev)
    ref = gq.gq_moe_decode(layer, x)
    need = gq.gq_moe_decode_workspace(layer, 6)
    pool = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=dev)   # NaN patterns
    rows = torch.full((8, 320), 7.0, dtype=torch.bfloat16, device=dev)
    y = gq.gq_moe_decode(layer, x, out=rows[1:7], workspace=pool[256:256 + need])
    torch.cuda.synchronize()
    assert torch.equal(y, ref)
    assert (rows[0] == 7).all() and (rows[7] == 7).all()
    assert (pool[:256] == 0xFF).all() and (pool[256 + need:] == 0xFF).all()
    with pytest.raises(gq.GQError):
        gq.gq_moe_decode(layer, x, workspace=pool[:need - 1])
    with pytest.raises(gq.GQError):
        gq.gq_moe_decode(layer, x, workspace=pool[1:])              # misaligned
    assert gq.gq_moe_decode(layer, x[:0]).shape == (0, 320)
    with pytest.raises(gq.GQError):
        gq.gq_moe_decode(layer, x.repeat(2, 1))                     # 12 tokens
    with pytest.raises(ValueError):
        gq.gq_moe_decode(layer, x[:, :256])
    with pytest.raises(ValueError):
        gq.gq_moe_decode(layer, x, out=rows)
    assert gq.gq_moe_decode_workspace(layer, 9) == -1


def test_two_graphs_share_a_workspace_between_eager_calls():
    """Two captured layers that use one workspace in turn, replayed with
    eager calls between, each replay equal to the eager result."""
    dev = device()
    cases = [Case("nf4", 10, 320, 128, 3), Case("mxfp4", 7, 288, 160, 4, bias=True)]
    layers = [c.layer(dev) for c in cases]
    xs = [to_dev_bf16(_x(c, r), dev) for c, r in zip(cases, (6, 3))]
    need = max(gq.gq_moe_decode_workspace(l, x.shape[0]) for l, x in zip(layers, xs))
    space = torch.empty(need, dtype=torch.uint8, device=dev)
    say("moe decode graphs")
    stream = torch.cuda.Stream()
    outs = [torch.empty_like(x) for x in xs]
    graphs = []
    with torch.cuda.stream(stream):
        for l, x, o in zip(layers, xs, outs):
            gq.gq_moe_decode(l, x, out=o, workspace=space)
        torch.cuda.synchronize()
        for l, x, o in zip(layers, xs, outs):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                gq.gq_moe_decode(l, x, out=o, workspace=space)
            graphs.append(g)
    for k in range(4):
        for x in xs:
            x.mul_(-1.0 if k % 2 else 0.5)
        eager = [gq.gq_moe_decode(l, x) for l, x in zip(layers, xs)]
        torch.cuda.synchronize()
        for o in outs:
            o.zero_()
        graphs[k % 2].replay()
        graphs[1 - k % 2].replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert torch.equal(o, e), k


def test_two_streams_at_once():
    dev = device()
    c = Case("nf4", 32, 1024, 512, 8)
    layer = c.layer(dev)
    x = to_dev_bf16(_x(c, 8), dev)
    say("moe decode two streams")
    ref = [gq.gq_moe_decode(layer, x), gq.gq_moe_decode(layer, x[:1])]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for k, part in ((0, x), (1, x[:1])):
            with torch.cuda.stream(s[k]):
                got[k].append(gq.gq_moe_decode(layer, part))
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(torch.equal(y, ref[k]) for y in got[k])


def test_weights_written_later_count():
    """The layer names its tensors; it holds no copy of them."""
    dev = device()
    c = Case("nf4", 6, 128, 64, 2)
    x = _x(c, 2)
    router = to_dev_bf16(c.router, dev)
    gu, dn = [tuple(to_dev(t, dev) for t in b) for b in (c.gu, c.dn)]
    layer = gq.gq_moe_layer(router, gu, dn, 2)
    say("moe decode weights written later")
    gq.gq_moe_decode(layer, to_dev_bf16(x, dev))
    dn[1].mul_(2)
    c.dn = (c.dn[0], c.dn[1] * 2)
    y = gq.gq_moe_decode(layer, to_dev_bf16(x, dev))
    torch.cuda.synchronize()
    c.check(y, x)


def test_layer_refuses_what_does_not_belong_together():
    dev = device()
    c = Case("nf4", 6, 128, 64, 2)
    router = to_dev_bf16(c.router, dev)
    gu, dn = [tuple(to_dev(t, dev) for t in b) for b in (c.gu, c.dn)]
    for bad in (dict(router=router[:, :64].contiguous()), dict(gu=dn), dict(dn=gu),
                dict(router_bias=router[0]), dict(down_bias=router.float()),
                dict(router=router.cpu())):
        a = dict(router=router, gu=gu, dn=dn)
        a.update({k: v for k, v in bad.items() if k in a})
        kw = {k: v for k, v in bad.items() if k not in a}
        with pytest.raises(ValueError):
            gq.gq_moe_layer(a["router"], a["gu"], a["dn"], 2, **kw)
    for topk in (0, 7):
        with pytest.raises(gq.GQError):
            gq.gq_moe_layer(router, gu, dn, topk)


def test_a_topk_past_32_bits_is_refused():
    dev = device()
    c = Case("nf4", 6, 128, 64, 2)
    gu, dn = [tuple(to_dev(t, dev) for t in b) for b in (c.gu, c.dn)]
    with pytest.raises(gq.GQError):
        gq.gq_moe_layer(to_dev_bf16(c.router, dev), gu, dn, (1 << 32) + 2)


def test_tensors_given_other_memory_leave_the_layer_as_it_was():
    dev = device()
    c = Case("nf4", 6, 128, 64, 2, bias=True)
    x = to_dev_bf16(_x(c, 3), dev)
    say("moe decode tensors given other memory")
    tensors = [to_dev_bf16(c.router, dev)] + [to_dev(t, dev) for t in (*c.gu, *c.dn)] + [
        to_dev_bf16(b, dev) for b in c.bias]
    layer = gq.gq_moe_layer(tensors[0], tensors[1:3], tensors[3:5], 2, router_bias=tensors[5],
                            gate_up_bias=tensors[6], down_bias=tensors[7])
    ref = gq.gq_moe_decode(layer, x)
    for t in tensors:
        t.data = torch.zeros_like(t)
    fill = [torch.full_like(t, 1) for t in tensors for _ in range(4)]    # takes what was freed
    y = gq.gq_moe_decode(layer, x)
    torch.cuda.synchronize()
    assert torch.equal(y, ref) and len(fill) == 32


class RandomCase(Case):
    """A layer of random bytes (made faster than packed weights)."""

    def __init__(self, fmt, E, H, I, topk, rows):
        g = np.random.default_rng([1, E, H, I, topk])
        self.fmt, self.E, self.H, self.I, self.topk, self.renorm = fmt, E, H, I, topk, rows % 2 == 0
        self.alpha, self.limit = 1.702, 7.0
        self.gu, self.dn = [self.bank(g, N, K) for N, K in ((2 * I, H), (H, I))]
        self.router = wl.draw_bf16(g, (E, H), std=0.1)
        self.bias = [wl.draw_bf16(g, s, std=0.5) for s in ((E,), (E, 2 * I), (E, H))]
        self.g = g

    def bank(self, g, N, K):
        codes = g.integers(0, 256, (self.E, N, K // 2), dtype=np.uint8)
        if self.fmt == "nf4":
            return codes, (0.02 + 0.04 * g.random((self.E, N, K // 64), dtype=np.float32))
        return (codes.reshape(self.E, N, K // 32, 16),
                g.integers(119, 122, (self.E, N, K // 32), dtype=np.uint8))


@pytest.mark.parametrize("fmt,E,H,I,topk,rows", [
    # one token, rows inside a wave, 8 and 4 rows a thread (64 slots: few columns suffice),
    # two and eight logits a lane
    ("nf4", 64, 1088, 512, 64, 1),
    ("nf4", 130, 1088, 512, 64, 1),
    ("nf4", 64, 1088, 256, 64, 1),
    ("nf4", 130, 1088, 256, 64, 1),
    ("nf4", 200, 128, 64, 5, 1),
    ("mxfp4", 64, 1056, 512, 64, 1),
    ("mxfp4", 130, 1056, 512, 64, 1),
    ("mxfp4", 64, 1056, 256, 64, 1),
    ("mxfp4", 130, 1056, 256, 64, 1),
    # rows that meet in LDS, 8, 4 and 2 a thread, three and one rows' segments a workgroup
    ("nf4", 9, 2112, 128, 8, 8),
    ("nf4", 130, 2112, 128, 8, 8),
    ("nf4", 9, 2112, 64, 8, 8),
    ("nf4", 130, 2112, 64, 8, 8),
    ("nf4", 130, 2112, 64, 2, 2),
    ("nf4", 3, 4160, 64, 2, 8),
    ("mxfp4", 130, 2080, 96, 8, 8),
    ("mxfp4", 9, 2080, 64, 8, 8),
    ("mxfp4", 130, 2080, 64, 8, 8),
    ("mxfp4", 130, 2080, 32, 2, 2),
    ("mxfp4", 3, 4128, 64, 2, 8),            # down: 2 steps, the last workgroup has one
    # down products of 4, 8 and 16 steps a workgroup, of 16 with a last one of 8
    ("nf4", 12, 2048, 768, 8, 8),
    ("nf4", 3, 2880, 1536, 2, 8),
    ("mxfp4", 3, 2880, 1536, 2, 8),
    ("mxfp4", 2, 4128, 1536, 1, 8),
    # two segments a lane in the down product, 8 and 16 steps
    ("nf4", 2, 2048, 2112, 2, 8),
    ("mxfp4", 2, 4128, 2080, 2, 8),
    ("mxfp4", 3, 2880, 2880, 2, 7),
])
def test_every_kernel_that_the_sizes_choose(fmt, E, H, I, topk, rows):
    dev = device()
    c = RandomCase(fmt, E, H, I, topk, rows)
    x = _x(c, rows)
    say("moe decode kernels", fmt, E, H, I, topk, rows)
    y = gq.gq_moe_decode(c.layer(dev), to_dev_bf16(x, dev))
    torch.cuda.synchronize()
    c.check(y, x)


def _choice_layer(dev, router, topk=1):
    """An MXFP4 layer whose output names the chosen expert: weights of zero
    and a down bias of e for expert e."""
    E, H = router.shape
    zeros = lambda *s: torch.zeros(s, dtype=torch.uint8, device=dev)          # noqa: E731
    bias = torch.arange(E, device=dev, dtype=torch.bfloat16).reshape(E, 1).expand(E, H).contiguous()
    return gq.gq_moe_layer(to_dev_bf16(router, dev), (zeros(E, 64, H // 32, 16), zeros(E, 64, H // 32)),
                           (zeros(E, H, 1, 16), zeros(E, H, 1)), topk, down_bias=bias)


@pytest.mark.parametrize("H,rows", [(64, 1), (64, 8), (544, 1), (2048, 8), (8192, 1), (8192, 8)])
def test_close_experts(H, rows):
    """Two experts whose logits differ by little more than the error that
    their sums may have: the larger one is chosen, and of equal ones the first.

    A lane adds at most H / 2048 pieces (rounded up) of four dot products; one
    is off by at most 3 2^-24 of the magnitudes that it adds (two roundings and
    the alignment of three terms); then 9 additions across lanes and waves and
    the bias's, half a step each.  So a logit is off by at most u = (12 pieces +
    10) 2^-24 of the sum of |x w|, and 2 u apart decides."""
    dev = device()
    for trial, x, pair, want in _close_pairs(H, rows):
        say("moe decode close experts", H, rows, trial, want)
        y = gq.gq_moe_decode(_choice_layer(dev, np.concatenate(pair)), to_dev_bf16(x, dev))
        torch.cuda.synchronize()
        assert (y.float().cpu() == want).all(), (trial, want)


def _close_pairs(H, rows):
    g = np.random.default_rng([H, rows])
    f = lambda b: oracle.bf16_to_f32(b).astype(np.float64)   # noqa: E731
    u = (12 * -(-H // 2048) + 10) * 2.0 ** -24
    for trial in range(12):
        x = wl.draw_bf16(g, (rows, H))
        w = wl.draw_bf16(g, (1, H), std=0.1)
        least = 2 * u * (np.abs(f(x)) @ np.abs(f(w[0]))).max()
        # one weight of the second expert one or a few steps larger in magnitude,
        # where every token has the same activation
        steps = np.arange(1, 129, dtype=np.uint16)[:, None]
        by = np.abs(f(x[0])) * np.abs(f(w + steps) - f(w))
        fits = np.argwhere((by > 1.3 * least) & (by < 2.6 * least))
        s, j = fits[g.integers(len(fits))]
        x[:, j] = x[0, j]
        up = w.copy()
        up[0, j] += s + 1
        gap = f(x[0])[j] * (f(up[0])[j] - f(w[0])[j])
        assert 2 * u * (np.abs(f(x)) @ np.abs(f(up[0]))).max() < abs(gap)
        yield trial, x, (w, up), int(gap > 0)
        yield trial, x, (up, w), int(gap < 0)
        yield trial, x, (w, w), 0


def test_subnormal_activations_and_weights_count():
    """bf16 subnormals of the token or of the router's weights: 2^-130 2^120 is
    a logit like any other."""
    dev = device()
    tiny, big = 0x0008, 0x7B80                               # 2^-130, 2^120
    say("moe decode subnormals")
    for x0, w0, w1 in ((tiny, big, big + 0x80), (big, tiny, 2 * tiny)):
        router = np.zeros((2, 64), dtype=np.uint16)
        router[:, 5] = w0, w1
        x = np.zeros((1, 64), dtype=np.uint16)
        x[0, 5] = x0
        y = gq.gq_moe_decode(_choice_layer(dev, router), to_dev_bf16(x, dev))
        torch.cuda.synchronize()
        assert (y.float().cpu() == 1).all()
