"""Timed cases of the root-mean-square norm with its residual addition, 8-bit
output and gradient, of the MXFP8 x MXFP4 grouped product, and of the expert
routing with groups, scores of either kind and a balancing bias.

``run`` computes a case with elementary torch operations, or, with ``own``
set, with this package's kernels; ``exact`` computes it again in 64 bits.
Sizes are the ones of the workloads this repository measures (hidden sizes of
2048 and 2880, experts of 2880 -> 5760 and 2880 -> 2880, 32 and 128 experts)
and generic and odd ones between them.
"""

import math

import torch

own = False

DEV = "cuda"
OSS_ALPHA, OSS_LIMIT = 1.702, 7.0
_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# e2m1 magnitudes by code
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    return [
        # the norm before the experts in one decode step: the residual stream is
        # added to, normed for the router and quantised for the experts
        dict(name="norm_step", op="norm", rows=4, H=2880, dtype="bf16", wdtype="bf16",
             residual=True, mxfp8=True, train=False, pad=0),
        # the same for a prefill
        dict(name="norm_prefill", op="norm", rows=8192, H=2880, dtype="bf16", wdtype="bf16",
             residual=True, mxfp8=True, train=False, pad=0),
        # rows of odd length cut out of a wider buffer, no residual, float32 gain
        dict(name="norm_odd", op="norm", rows=1333, H=1023, dtype="f16", wdtype="f32",
             residual=False, mxfp8=False, train=False, pad=9),
        # a training step: the norm and its gradient, which joins the residual's
        dict(name="norm_train", op="norm", rows=16384, H=2048, dtype="bf16", wdtype="bf16",
             residual=True, mxfp8=False, train=True, pad=0),
        # one token through four experts' gate_up with the gated unit
        dict(name="product_step", op="product", rows=1, topk=4, E=32, N=5760, K=2880, unit=True,
             weights=False, dropped=0.0),
        # odd sizes: widths that end inside a tile, a K tail, few rows per expert, dropped pairs
        dict(name="product_ragged", op="product", rows=333, topk=2, E=6, N=544, K=1056, unit=False,
             weights=True, dropped=0.05),
        # a prefill's gate_up with the gated unit: 2048 tokens, 4 of 32 experts
        dict(name="product_gate_up", op="product", rows=2048, topk=4, E=32, N=5760, K=2880,
             unit=True, weights=False, dropped=0.0),
        # its down product: one row per (token, expert) pair, router weights applied
        dict(name="product_down", op="product", rows=8192, topk=1, E=32, N=2880, K=2880,
             unit=False, weights=True, dropped=0.0),
        # routing of one decode step: sigmoid scores, balancing bias, 4 of 8 groups
        dict(name="route_step", op="route", rows=4, E=256, topk=8, dtype="f32", score="sigmoid",
             bias=True, groups=8, topk_groups=4, group_top=2, renorm=True, scale=2.5,
             train=False, masked=False),
        # the same for a prefill's tokens
        dict(name="route_prefill", op="route", rows=16384, E=256, topk=8, dtype="f32",
             score="sigmoid", bias=True, groups=8, topk_groups=4, group_top=2, renorm=True,
             scale=2.5, train=False, masked=False),
        # routing and its gradient in a training step, no groups; some experts masked
        dict(name="route_train", op="route", rows=16384, E=128, topk=8, dtype="bf16",
             score="sigmoid", bias=True, groups=1, topk_groups=1, group_top=1, renorm=True,
             scale=1.0, train=True, masked=True),
        # groups of an odd size by their best expert, softmax scores as they are
        dict(name="route_odd", op="route", rows=1000, E=60, topk=6, dtype="f16", score="softmax",
             bias=False, groups=12, topk_groups=3, group_top=1, renorm=False, scale=16.0,
             train=True, masked=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "product", "route"])
    if op == "norm":
        train = rng.random() < 0.4
        mxfp8 = not train and rng.random() < 0.6
        # (a row of one value has a gradient of nearly nothing, which 32 bits cannot hold)
        H = 32 * _log_int(rng, 1, 256) if mxfp8 else _log_int(rng, 8 if train else 1, 8192)
        return dict(op=op, rows=_log_int(rng, 1, min(16384, 8192 * 2880 // H)), H=H,
                    dtype=rng.choice(sorted(_DT)) if not mxfp8 else rng.choice(["bf16", "f16"]),
                    wdtype=rng.choice(["same", "f32"]), residual=rng.random() < 0.6, mxfp8=mxfp8,
                    train=train, pad=rng.choice([0, 0, 1, 7, 8, 64]))
    if op == "product":
        E = rng.randint(1, 32)
        topk = rng.randint(1, min(4, E))
        unit = rng.random() < 0.5
        return dict(op=op, rows=_log_int(rng, 1, 8192 // topk), topk=topk, E=E,
                    N=32 * rng.randint(1, 150), K=32 * rng.randint(1, 90), unit=unit,
                    weights=not unit and rng.random() < 0.5, dropped=rng.choice([0.0, 0.1]))
    groups = rng.choice([1, 1, 2, 4, 8, 8, 16])
    size = rng.randint(1 if groups > 1 else 2, 320 // groups)
    topk_groups = rng.randint(1, groups)
    return dict(op="route", rows=_log_int(rng, 1, 16384), E=groups * size,
                topk=rng.randint(1, min(10, topk_groups * size)), dtype=rng.choice(sorted(_DT)),
                score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, groups=groups,
                topk_groups=topk_groups, group_top=rng.choice([1, 2]),
                renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5, 16.0]),
                train=rng.random() < 0.5, masked=rng.random() < 0.4)


# ---- inputs -----------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _mx_bank(g, E, N, K):
    blocks = torch.randint(0, 256, (E, N, K // 32, 16), dtype=torch.uint8, device=DEV, generator=g)
    scales = torch.randint(119, 122, (E, N, K // 32), dtype=torch.uint8, device=DEV, generator=g)
    return blocks, scales


def _topk_ids(g, rows, E, topk, dropped):
    ids = torch.rand((rows, E), device=DEV, generator=g).argsort(dim=1)[:, :topk].to(torch.int32)
    if dropped:
        ids = torch.where(torch.rand((rows, topk), device=DEV, generator=g) < dropped, -1, ids)
    return ids.to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op == "norm":
        rows, H, dt = case["rows"], case["H"], _DT[case["dtype"]]
        wide = H + case["pad"]
        # a residual stream with outlier channels, and what a layer adds to it
        spread = torch.exp2(torch.randint(-1, 4, (1, wide), generator=g, device=DEV).float())
        s["x"] = (torch.randn((rows, wide), generator=g, device=DEV) * spread).to(dt)[:, :H]
        s["residual"] = _randn(g, rows, H, std=2.0, dtype=dt) if case["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(
            dt if case["wdtype"] == "same" else _DT[case["wdtype"]])
        if case["train"]:
            s["d_y"] = _randn(g, rows, H, std=0.1, dtype=dt)
            s["d_residual"] = _randn(g, rows, H, std=0.1, dtype=dt) if case["residual"] else None
    elif op == "product":
        s["x"] = _randn(g, case["rows"], case["K"], dtype=torch.bfloat16)
        s["blocks"], s["scales"] = _mx_bank(g, case["E"], case["N"], case["K"])
        s["ids"] = _topk_ids(g, case["rows"], case["E"], case["topk"], case["dropped"])
        pairs = case["rows"] * case["topk"]
        s["weights"] = torch.rand(pairs, generator=g, device=DEV) if case["weights"] else None
    else:
        rows, E = case["rows"], case["E"]
        z = torch.randn((rows, E), generator=g, device=DEV) * 1.5
        if case["masked"]:             # experts that a token may not take; a few rows have none
            z = z.masked_fill(torch.rand((rows, E), generator=g, device=DEV) < 0.2, -math.inf)
            z = z.masked_fill(torch.rand((rows, 1), generator=g, device=DEV) < 0.02, -math.inf)
        s["logits"] = z.to(_DT[case["dtype"]])
        s["bias"] = _randn(g, E, std=0.1) if case["bias"] else None
        s["d_weights"] = _randn(g, rows, case["topk"])
    return s


EPS = 1e-6


# ---- plain forms --------------------------------------------------------------
def _norm(s):
    c = s["case"]
    dt = s["x"].dtype
    got = {}
    h = s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(dt)
        got["residual"] = h
    v = h.float()
    rstd = 1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    w = s["weight"].float()
    y = v * rstd * w
    got["y"] = y.to(dt)
    if c["mxfp8"]:
        got["values"] = _quantize8(y).to(torch.bfloat16)
    if c["train"]:
        # y = n w, n = h rstd:  dh = rstd (g - n mean(g n)), g = dy w;  dw = sum of dy n
        dy = s["d_y"].float()
        n = v * rstd
        gw = dy * w
        dx = rstd * (gw - n * (gw * n).mean(dim=1, keepdim=True))
        if s["d_residual"] is not None:
            dx = dx + s["d_residual"].float()
        got["d_x"] = dx.to(dt)
        got["d_weight"] = (dy * n).sum(dim=0).to(s["weight"].dtype)
    return got


def _quantize8(x):
    """MXFP8 of x [rows, K]: the values that the codes and scales stand for, float32."""
    rows, K = x.shape
    b = x.float().reshape(rows, K // 32, 32)
    m, e = torch.frexp(b.abs().amax(dim=-1, keepdim=True))
    # the least X with amax 2^-X <= 448
    X = torch.where(m > 0, e - 9 + (m > 0.875).int(), -127).clamp(-127, 127)
    v = torch.ldexp(b.abs(), -X)
    step = torch.ldexp(torch.ones_like(v), (torch.frexp(v).exponent - 1).clamp(min=-6) - 3)
    v = torch.round(v / step) * step                           # half to even
    return torch.ldexp(torch.copysign(v, b), X).reshape(rows, K)


def _mx_values(blocks, scales):
    table = torch.tensor(E2M1 + [-v for v in E2M1], device=blocks.device)
    codes = torch.stack([blocks & 15, blocks >> 4], dim=-1).flatten(-2)
    v = table[codes.int()] * torch.exp2(scales.float() - 127).unsqueeze(-1)
    return v.flatten(-2)


def _oss_unit(gate, up):
    gate, up = gate.clamp(max=OSS_LIMIT), up.clamp(-OSS_LIMIT, OSS_LIMIT)
    return gate / (1 + torch.exp(-OSS_ALPHA * gate)) * (up + 1)


def _product(s):
    c = s["case"]
    rows, topk, E = c["rows"], c["topk"], c["E"]
    x = _quantize8(s["x"])
    flat = s["ids"].reshape(-1).long()
    token = torch.arange(rows * topk, device=flat.device) // topk
    if rows * topk <= 8:                                   # one product per pair
        live = ((flat >= 0) & (flat < E)).float()
        at = flat.clamp(0, E - 1)
        W = _mx_values(s["blocks"][at], s["scales"][at])
        y = torch.matmul(W, x[token].unsqueeze(-1)).squeeze(-1) * live.unsqueeze(1)
    else:
        # rows grouped by expert, each group filled up to the longest
        key = torch.where((flat >= 0) & (flat < E), flat, E)
        order = torch.argsort(key, stable=True)
        count = torch.bincount(key, minlength=E + 1)
        place = torch.arange(rows * topk, device=flat.device) - (count.cumsum(0) - count)[key[order]]
        cap = int(count.max())
        grouped = x.new_zeros(E + 1, c["K"], cap)
        grouped[key[order], :, place] = x[token[order]]
        W = _mx_values(s["blocks"], s["scales"])
        out = torch.matmul(W, grouped[:E])                 # [E, N, cap]
        out = torch.cat([out, out.new_zeros(1, c["N"], cap)])
        y = torch.empty(rows * topk, c["N"], device=flat.device)
        y[order] = out[key[order], :, place]
    if c["unit"]:
        live = ((flat >= 0) & (flat < E)).unsqueeze(1)
        y = torch.where(live, _oss_unit(y[:, 0::2], y[:, 1::2]), 0.0)
    if s["weights"] is not None:
        y = y * s["weights"].unsqueeze(1)
    return y.to(torch.bfloat16)


def _scores(z, score):
    """Scores in 64 bits (two experts at the border of the selection may be
    close); a row without a live expert has zeros."""
    z = z.double()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    peak = z.amax(dim=1, keepdim=True)
    p = torch.exp(z - torch.where(peak > -math.inf, peak, 0.0))
    total = p.sum(dim=1, keepdim=True)
    return p / torch.where(total > 0, total, 1.0)


def _route(s):
    c = s["case"]
    z, topk, groups = s["logits"].double(), c["topk"], c["groups"]
    rows, E = z.shape
    score = _scores(s["logits"], c["score"])
    dead = z == -math.inf
    # without a bias the scores' order is the logits'
    choice = z if s["bias"] is None else score + s["bias"].double()
    choice = torch.where(dead, -math.inf, choice)
    if groups > 1:
        # a group counts as its best expert, or as its two best's scores together
        best = choice
        if c["group_top"] == 2 and s["bias"] is None:
            best = torch.where(dead, -math.inf, score)
        best = best.reshape(rows, groups, E // groups)
        best = torch.sort(best, dim=2, descending=True).values[..., :c["group_top"]]
        first = best[..., 0]
        rest = torch.where(best[..., 1:] > -math.inf, best[..., 1:], 0.0).sum(dim=2)
        order = torch.sort(first + rest, dim=1, descending=True, stable=True).indices
        keep = torch.zeros_like(first, dtype=torch.bool)
        keep = keep.scatter(1, order[:, :c["topk_groups"]], True)
        choice = torch.where(keep.repeat_interleave(E // groups, dim=1), choice, -math.inf)
    top, ids = torch.sort(choice, dim=1, descending=True, stable=True)
    live = top[:, :topk] > -math.inf
    ids = ids[:, :topk]
    w = torch.where(live, score.gather(1, ids), 0.0)
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    ids = torch.where(live, ids, -1).to(torch.int32)
    return ids, (w * c["scale"]).float()


def _route_backward(s, ids):
    c = s["case"]
    live = ids >= 0
    at = torch.where(live, ids, 0).long()
    score = _scores(s["logits"], c["score"]).float()
    p = torch.where(live, score.gather(1, at), 0.0)        # the chosen scores
    g = torch.where(live, s["d_weights"] * c["scale"], 0.0)
    if c["renorm"]:
        total = p.sum(dim=1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        g = (g - (g * p).sum(dim=1, keepdim=True) / total) / total
        g = torch.where(live, g, 0.0)
    if c["score"] == "sigmoid":
        grad = torch.zeros_like(score).scatter_add(1, at, g * p * (1 - p))
    else:
        grad = torch.zeros_like(score).scatter_add(1, at, g * p)
        grad = grad - score * (g * p).sum(dim=1, keepdim=True)
    return grad.to(s["logits"].dtype)


# ---- one pass -------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "norm":
        return _norm(state)
    if c["op"] == "product":
        return {"y": _product(state)}
    ids, weights = _route(state)
    got = {"ids": ids, "weights": weights}
    if c["train"]:
        got["d_logits"] = _route_backward(state, ids)
    return got


def _run_own(s):
    import bit_grouped_moe_amd as gq
    c = s["case"]
    if c["op"] == "norm":
        got = {}
        # codes, scales and the values they stand for come from the same launch
        n = gq.gq_rms_norm(s["x"], s["weight"], eps=EPS, residual=s["residual"], mxfp8=c["mxfp8"],
                           values=c["mxfp8"])
        got["y"] = n.y
        if s["residual"] is not None:
            got["residual"] = n.residual
        if c["mxfp8"]:
            got["values"] = n.values
        if c["train"]:
            h = s["x"] if s["residual"] is None else n.residual
            got["d_x"], got["d_weight"] = gq.gq_rms_norm_backward(
                s["d_y"], h, s["weight"], eps=EPS, d_residual=s["d_residual"])
        return got
    if c["op"] == "product":
        x = gq.gq_mxfp8_quantize(s["x"])
        if c["rows"] <= 8:
            if c["unit"]:
                y = gq.gq_mxfp4_grouped_gemv_fp8_swiglu(x, s["blocks"], s["scales"], s["ids"])
            else:
                y = gq.gq_mxfp4_grouped_gemv_fp8(x, s["blocks"], s["scales"], s["ids"],
                                                 pair_scale=s["weights"])
            return {"y": y}
        route = gq.gq_route_sort(s["ids"], c["E"])
        if c["unit"]:
            y = gq.gq_mxfp4_grouped_gemm_fp8_swiglu(x, s["blocks"], s["scales"], route)
        else:
            y = gq.gq_mxfp4_grouped_gemm_fp8(x, s["blocks"], s["scales"], route,
                                             pair_scale=s["weights"])
        return {"y": y}
    ids, weights = gq.gq_moe_route(s["logits"], c["topk"], score=c["score"], bias=s["bias"],
                                   groups=c["groups"], topk_groups=c["topk_groups"],
                                   group_top=c["group_top"], renormalize=c["renorm"],
                                   scale=c["scale"])
    got = {"ids": ids, "weights": weights}
    if c["train"]:
        got["d_logits"] = gq.gq_moe_route_backward(s["d_weights"], s["logits"], ids,
                                                   score=c["score"], renormalize=c["renorm"],
                                                   scale=c["scale"])
    return got


# ---- what a pass cannot do without ---------------------------------------------------
def work(case):
    c = case
    if c["op"] == "norm":
        size = 4 if c["dtype"] == "f32" else 2
        n = c["rows"] * c["H"]
        b = n * size * (4 if c["residual"] else 2)             # x, residual; their sum, y
        if c["mxfp8"]:                                         # codes, scales and their values
            b += n * (1 + 1 / 32 + 2)
        if c["train"]:                                         # d_y, the sum; d_x
            b += n * size * (4 if c["residual"] else 3)
        return {"bytes": b + 4 * c["H"], "flops": n * (5 + (10 if c["train"] else 0))}
    if c["op"] == "product":
        pairs = c["rows"] * c["topk"]
        used = min(c["E"], pairs) if c["rows"] > 1 else c["topk"]
        out = c["N"] // 2 if c["unit"] else c["N"]
        return {"bytes": c["rows"] * c["K"] * 2 + used * c["N"] * c["K"] * (0.5 + 1 / 32)
                + pairs * out * 2, "flops": 2 * pairs * c["N"] * c["K"]}
    size = 4 if c["dtype"] == "f32" else 2
    n, k = c["rows"] * c["E"], c["rows"] * c["topk"]
    b = n * size + k * 8
    if c["train"]:
        b += n * size * 2 + k * 8
    return {"bytes": b, "flops": 6 * n * (2 if c["train"] else 1)}


# ---- from the definitions, in 64 bits ----------------------------------------------------
def _norm64(s):
    c = s["case"]
    x, w = s["x"].double(), s["weight"].double()
    got = {}
    if s["residual"] is not None:
        # the sum is kept in the stream's type, and the norm is the norm of what is kept
        x = (x + s["residual"].double()).to(s["x"].dtype).double()
        got["residual"] = x
    root = torch.linalg.vector_norm(x, dim=1, keepdim=True) / math.sqrt(c["H"])
    root = torch.hypot(root, root.new_tensor(math.sqrt(EPS)))
    got["y"] = x / root * w
    if c["mxfp8"]:
        # next to the border of two 8-bit values the last bit of the norm decides,
        # so that no value here is right for every order of a sum
        got["values"] = None
    if c["train"]:
        dy = s["d_y"].double()
        got["d_weight"] = (x / root * dy).sum(dim=0)
        # dL/dx_i = dy_i w_i / r - x_i / (H r^3) sum_j dy_j w_j x_j
        dot = (dy * w * x).sum(dim=1, keepdim=True)
        d = dy * w / root - x * dot / (c["H"] * root ** 3)
        got["d_x"] = d if s["d_residual"] is None else d + s["d_residual"].double()
    return got


def _q64(x):
    """The nearest e4m3 value by search in the table, an even code where two are equally near."""
    code = torch.arange(127, device=x.device)
    e, m = code // 8, (code % 8).double()
    table = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    b = x.double().reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(dim=-1, keepdim=True)
    X = torch.ceil(torch.log2(amax / 448)).clamp(-127, 127)
    # the logarithm may be off at a power of two
    X = torch.where(amax * torch.exp2(-(X - 1)) <= 448, X - 1, X)
    X = torch.where(amax * torch.exp2(-X) > 448, X + 1, X)
    scale = torch.exp2(torch.where(amax > 0, X, -127.0))
    v = b.abs() / scale
    hi = torch.searchsorted(table, v).clamp(max=126)           # the first value >= v
    lo = (hi - 1).clamp(min=0)
    down, up = v - table[lo], table[hi] - v
    near = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return (torch.copysign(table[near], b) * scale).reshape(x.shape)


def _w64(blocks, scales):
    n = blocks.shape[0]
    a = blocks.reshape(n, -1).long()
    t = torch.tensor(E2M1 + [-m for m in E2M1], dtype=torch.float64, device=a.device)
    v = torch.empty((n, a.shape[1] * 2), dtype=torch.float64, device=a.device)
    v[:, 0::2], v[:, 1::2] = t[a % 16], t[a // 16]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1)


def _unit64(h):
    gate = torch.minimum(h[..., 0::2], h.new_tensor(OSS_LIMIT))
    up = torch.clip(h[..., 1::2], -OSS_LIMIT, OSS_LIMIT)
    return gate * torch.sigmoid(OSS_ALPHA * gate) * (up + 1)


def _largest(v, count):
    """count times the largest that is left of each row, the first of equal
    ones: (places, -1 where only -inf is left)."""
    left, places = v.clone(), []
    for _ in range(count):
        most = left.amax(dim=1, keepdim=True)
        at = (left == most).to(torch.int8).argmax(dim=1, keepdim=True)
        places.append(torch.where(most == -math.inf, -1, at))
        left = left.scatter(1, at, -math.inf)
    return torch.cat(places, dim=1)


def _route64(s):
    c = s["case"]
    z, G = s["logits"].double(), c["groups"]
    rows, E = z.shape
    some = (z > -math.inf).any(dim=1, keepdim=True)
    if c["score"] == "sigmoid":
        logp = torch.nn.functional.logsigmoid(z)
    else:
        logp = torch.log_softmax(torch.where(some, z, 0.0), dim=1)
    value = torch.exp(logp) if s["bias"] is None else torch.exp(logp) + s["bias"].double()
    value = torch.where(z == -math.inf, -math.inf, value)
    order = value if s["bias"] is not None else z
    if G > 1:
        v = (order if c["group_top"] == 1 else value).reshape(rows * G, E // G)
        two = _largest(v, min(c["group_top"], E // G))
        v = torch.where(two >= 0, v.gather(1, two.clamp(min=0)), 0.0).sum(dim=1)
        v = torch.where(two[:, 0] >= 0, v, -math.inf).reshape(rows, G)
        chosen = _largest(v, c["topk_groups"])
        open_ = torch.zeros((rows, G + 1), dtype=torch.bool, device=z.device)
        open_ = open_.scatter(1, torch.where(chosen >= 0, chosen, G), True)[:, :G]
        order = torch.where(open_[:, torch.arange(E, device=z.device) // (E // G)], order, -math.inf)
    ids = _largest(order, c["topk"])
    live = ids >= 0
    lw = torch.where(live, logp.gather(1, ids.clamp(min=0)), -math.inf)
    if c["renorm"]:
        norm = torch.logsumexp(torch.where(live[:, :1], lw, 0.0), dim=1, keepdim=True)
        lw = lw - norm
    weights = torch.where(live, torch.exp(lw), 0.0) * c["scale"]
    got = {"ids": None, "weights": weights}
    if c["train"]:
        # the derivative of log weight by log weight: w_s (1 - w) sums, slot by slot
        w = weights / c["scale"]
        d = torch.where(live, s["d_weights"].double(), 0.0) * c["scale"]
        up = d * w                                         # by each chosen log score
        if c["renorm"]:
            up = up - w * (d * w).sum(dim=1, keepdim=True)
        wide = torch.zeros((rows, E + 1), dtype=torch.float64, device=z.device)
        wide = wide.scatter_add(1, torch.where(live, ids, E), up)[:, :E]
        if c["score"] == "sigmoid":
            got["d_logits"] = wide * torch.sigmoid(-z)     # d log sigmoid(z) / dz
        else:
            p = torch.where(some, torch.exp(logp), 0.0)
            got["d_logits"] = wide - p * wide.sum(dim=1, keepdim=True)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        return _norm64(s)
    if c["op"] == "product":
        x = _q64(s["x"])
        flat = s["ids"].reshape(-1)
        out = c["N"] // 2 if c["unit"] else c["N"]
        y = torch.zeros((flat.numel(), out), dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            at = (flat == e).nonzero().reshape(-1)
            if at.numel():
                h = x[at // c["topk"]] @ _w64(s["blocks"][e], s["scales"][e]).t()
                y[at] = _unit64(h) if c["unit"] else h
        if s["weights"] is not None:
            y *= s["weights"].double()[:, None]
        return {"y": y}
    return _route64(s)
