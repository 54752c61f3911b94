"""Timed cases of the MXFP4 quantiser, the MXFP4 x MXFP4 grouped product, the
expert router and the whole mixture-of-experts layer for a few tokens.

``run`` computes a case with elementary torch operations, or, with ``own``
set, with this package's kernels; ``exact`` computes it again in 64 bits.
Sizes are the ones of the two workloads this repository measures (experts
of 2048 -> 1536/768 -> 2048 weights in NF4, 2880 -> 5760/2880 -> 2880 in
MXFP4) and odd ones between them.
"""

import math

import torch

own = False

DEV = "cuda"
OSS_ALPHA, OSS_LIMIT = 1.702, 7.0
_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# e2m1 magnitudes by code, and the NF4 data type of QLoRA (Dettmers et al. 2023)
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
NF4_BITS = [0xBF800000, 0xBF3239B1, 0xBF066B30, 0xBECA32A0, 0xBE91A24D, 0xBE3D353F, 0xBDBA7871, 0,
            0x3DA2FAFF, 0x3E24CAE3, 0x3E7C04DD, 0x3EAD033A, 0x3EE1A4B8, 0x3F1007AB, 0x3F3913B3,
            0x3F800000]


def listed():
    return [
        # one decode step's activations on their way into a 4-bit product
        dict(name="quantize_step", op="quantize", rows=4, K=2880, dtype="bf16", pad=0),
        # a prefill's expert activations, 2048 tokens x 4 experts, rows cut out of a wider buffer
        dict(name="quantize_prefill", op="quantize", rows=8192, K=2880, dtype="bf16", pad=64),
        # float32 master weights of eight experts' gate_up packed on the device
        dict(name="quantize_weights", op="quantize", rows=46080, K=2880, dtype="f32", pad=0),
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
        # a whole layer for one token, NF4 experts
        dict(name="layer_nf4_one", op="layer", fmt="nf4", rows=1, topk=8, E=128, H=2048, I=768,
             bias=False, renorm=True),
        # a whole layer for one token, MXFP4 experts with their biases
        dict(name="layer_mxfp4_one", op="layer", fmt="mxfp4", rows=1, topk=4, E=32, H=2880, I=2880,
             bias=True, renorm=True),
        # eight tokens of a small serving batch
        dict(name="layer_nf4_eight", op="layer", fmt="nf4", rows=8, topk=8, E=128, H=2048, I=768,
             bias=False, renorm=True),
        # routing of one decode step's tokens
        dict(name="route_step", op="route", rows=4, E=128, topk=8, dtype="f32", renorm=True,
             train=False, masked=False),
        # routing and its gradient in a training step; some experts masked
        dict(name="route_train", op="route", rows=16384, E=128, topk=8, dtype="bf16", renorm=True,
             train=True, masked=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "layer", "route"])
    if op == "quantize":
        K = 32 * rng.randint(1, 180)
        rows = min(_log_int(rng, 1, 40000), 46080 * 2880 // K)
        return dict(op=op, rows=rows, K=K, dtype=rng.choice(sorted(_DT)),
                    pad=rng.choice([0, 0, 1, 7, 8, 64]))
    if op == "product":
        E = rng.randint(1, 32)
        topk = rng.randint(1, min(4, E))
        unit = rng.random() < 0.5
        return dict(op=op, rows=_log_int(rng, 1, 8192 // topk), topk=topk, E=E,
                    N=32 * rng.randint(1, 150), K=32 * rng.randint(1, 90), unit=unit,
                    weights=not unit and rng.random() < 0.5, dropped=rng.choice([0.0, 0.1]))
    if op == "layer":
        E = rng.randint(2, 128)
        topk = rng.randint(1, min(8, E))
        fmt = rng.choice(["nf4", "mxfp4"])
        unit = 64 if fmt == "nf4" else 32
        top = 2048 if E > 40 else 2880
        return dict(op=op, fmt=fmt, rows=rng.randint(1, 8), topk=topk, E=E,
                    H=unit * rng.randint(2, top // unit), I=unit * rng.randint(2, 1536 // unit),
                    bias=rng.random() < 0.5, renorm=rng.random() < 0.7)
    E = rng.randint(1, 320)
    return dict(op="route", rows=_log_int(rng, 1, 16384), E=E, topk=rng.randint(1, min(10, E)),
                dtype=rng.choice(sorted(_DT)), renorm=rng.random() < 0.6,
                train=rng.random() < 0.5, masked=rng.random() < 0.5)


# ---- inputs -----------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _nf4_bank(g, E, N, K):
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    # the largest of 64 normal draws of standard deviation 0.02
    absmax = 0.02 * (2.0 + torch.rand((E, N, K // 64), device=DEV, generator=g))
    return codes, absmax


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
    if op == "quantize":
        rows, K = case["rows"], case["K"]
        # activations with outlier channels: a block's values span several powers of two
        x = torch.randn((rows, K + case["pad"]), generator=g, device=DEV)
        x *= torch.exp2(torch.randint(-2, 4, (1, K + case["pad"]), generator=g, device=DEV).float())
        s["x"] = x.to(_DT[case["dtype"]])[:, :K]
    elif op == "product":
        s["x"] = _randn(g, case["rows"], case["K"], dtype=torch.bfloat16)
        s["blocks"], s["scales"] = _mx_bank(g, case["E"], case["N"], case["K"])
        s["ids"] = _topk_ids(g, case["rows"], case["E"], case["topk"], case["dropped"])
        pairs = case["rows"] * case["topk"]
        s["weights"] = torch.rand(pairs, generator=g, device=DEV) if case["weights"] else None
    elif op == "layer":
        E, H, I = case["E"], case["H"], case["I"]
        bank = _nf4_bank if case["fmt"] == "nf4" else _mx_bank
        s["x"] = _randn(g, case["rows"], H, dtype=torch.bfloat16)
        s["router"] = _randn(g, E, H, std=0.05, dtype=torch.bfloat16)
        s["gate_up"] = bank(g, E, 2 * I, H)
        s["down"] = bank(g, E, H, I)
        b = case["bias"]
        s["router_bias"] = _randn(g, E, std=0.5, dtype=torch.bfloat16) if b else None
        s["gate_up_bias"] = _randn(g, E, 2 * I, std=0.5, dtype=torch.bfloat16) if b else None
        s["down_bias"] = _randn(g, E, H, std=0.5, dtype=torch.bfloat16) if b else None
        if own:                        # the layer's weights, checked once as a program does at load
            import bit_grouped_moe_amd as gq
            s["layer"] = gq.gq_moe_layer(s["router"], s["gate_up"], s["down"], case["topk"],
                                         router_bias=s["router_bias"],
                                         gate_up_bias=s["gate_up_bias"],
                                         down_bias=s["down_bias"], renormalize=case["renorm"])
    else:
        rows, E = case["rows"], case["E"]
        z = torch.randn((rows, E), generator=g, device=DEV) * 2
        if case["masked"]:             # experts that a token may not take; a few rows have none
            z = z.masked_fill(torch.rand((rows, E), generator=g, device=DEV) < 0.2, -math.inf)
            z = z.masked_fill(torch.rand((rows, 1), generator=g, device=DEV) < 0.02, -math.inf)
        s["logits"] = z.to(_DT[case["dtype"]])
        s["d_weights"] = _randn(g, rows, case["topk"])
    return s


# ---- plain forms --------------------------------------------------------------
def _quantize(x):
    """MXFP4 of x [rows, K]: the values that the codes and scales stand for, float32."""
    rows, K = x.shape
    b = x.float().reshape(rows, K // 32, 32)
    amax = b.abs().amax(dim=-1, keepdim=True)
    X = (torch.frexp(amax).exponent - 3).clamp(-127, 127)      # floor(log2 amax) - 2
    m = torch.ldexp(b.abs(), -X)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    m = (torch.round(m / step) * step).clamp(max=6.0)          # half to even
    return torch.ldexp(torch.copysign(m, b), X).reshape(rows, K)


def _mx_values(blocks, scales):
    table = torch.tensor(E2M1 + [-v for v in E2M1], device=blocks.device)
    codes = torch.stack([blocks & 15, blocks >> 4], dim=-1).flatten(-2)
    v = table[codes.int()] * torch.exp2(scales.float() - 127).unsqueeze(-1)
    return v.flatten(-2)


def _nf4_values(codes, absmax):
    table = torch.tensor(NF4_BITS, dtype=torch.int64).to(torch.int32).view(torch.float32)
    q = torch.stack([codes >> 4, codes & 15], dim=-1).flatten(-2)
    v = table.to(codes.device)[q.int()].unflatten(-1, (-1, 64))
    return (v * absmax.unsqueeze(-1)).flatten(-2)


def _oss_unit(gate, up):
    gate, up = gate.clamp(max=OSS_LIMIT), up.clamp(-OSS_LIMIT, OSS_LIMIT)
    return gate / (1 + torch.exp(-OSS_ALPHA * gate)) * (up + 1)


def _select(logits, topk, renorm):
    """The topk largest logits of each row, ties to the lower index; a
    slot that only masked experts (-inf) are left for is id -1, weight 0."""
    z = logits.float() if logits.dtype != torch.float64 else logits
    top, ids = torch.sort(z, dim=1, descending=True, stable=True)
    top, ids = top[:, :topk], ids[:, :topk]
    live = top > -math.inf
    peak = torch.where(live[:, :1], top[:, :1], 0.0)
    part = torch.exp(top - peak)
    total = (part if renorm else torch.exp(z - peak)).sum(dim=1, keepdim=True)
    weights = torch.where(live, part / torch.where(total > 0, total, 1.0), 0.0)
    return torch.where(live, ids, -1).to(torch.int32), weights


def _select_backward(d_weights, logits, ids, weights, renorm):
    live = ids >= 0
    dot = (d_weights * weights).sum(dim=1, keepdim=True)
    z = logits.float()
    # one more column takes what the dead slots would add
    grad = z.new_zeros(z.shape[0], z.shape[1] + 1)
    at = torch.where(live, ids, z.shape[1]).long()
    if renorm:
        grad = grad.scatter_add(1, at, weights * (d_weights - dot))[:, :-1]
    else:
        peak = z.amax(dim=1, keepdim=True)
        p = torch.exp(z - torch.where(peak > -math.inf, peak, 0.0))
        total = p.sum(dim=1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
        grad = p * (grad.scatter_add(1, at, torch.where(live, d_weights, 0.0))[:, :-1] - dot)
    return grad.to(logits.dtype)


def _product(s):
    c = s["case"]
    rows, topk, E = c["rows"], c["topk"], c["E"]
    x = _quantize(s["x"])
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


def _layer(s):
    c = s["case"]
    x = s["x"].float()
    # in 64 bits: two experts at the border of the selection may be close
    logits = s["x"].double() @ s["router"].double().t()
    if s["router_bias"] is not None:
        logits = logits + s["router_bias"].double()
    ids, weights = _select(logits, c["topk"], c["renorm"])
    flat = ids.reshape(-1).long()
    token = torch.arange(flat.numel(), device=x.device) // c["topk"]
    values = _nf4_values if c["fmt"] == "nf4" else _mx_values
    h = torch.matmul(values(s["gate_up"][0][flat], s["gate_up"][1][flat]),
                     x[token].unsqueeze(-1)).squeeze(-1)
    if s["gate_up_bias"] is not None:
        h = h + s["gate_up_bias"][flat].float()
    if c["fmt"] == "nf4":
        gate, up = h[:, :c["I"]], h[:, c["I"]:]
        act = gate / (1 + torch.exp(-gate)) * up
    else:
        act = _oss_unit(h[:, 0::2], h[:, 1::2])
    y = torch.matmul(values(s["down"][0][flat], s["down"][1][flat]), act.unsqueeze(-1)).squeeze(-1)
    if s["down_bias"] is not None:
        y = y + s["down_bias"][flat].float()
    y = y * weights.float().reshape(-1, 1)
    return y.reshape(c["rows"], c["topk"], c["H"]).sum(dim=1).to(torch.bfloat16)


# ---- one pass -------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "quantize":
        return {"values": _quantize(state["x"]).to(torch.bfloat16)}
    if c["op"] == "product":
        return {"y": _product(state)}
    if c["op"] == "layer":
        return {"y": _layer(state)}
    ids, weights = _select(state["logits"], c["topk"], c["renorm"])
    got = {"ids": ids, "weights": weights}
    if c["train"]:
        got["d_logits"] = _select_backward(state["d_weights"], state["logits"], ids, weights,
                                           c["renorm"])
    return got


def _run_own(s):
    import bit_grouped_moe_amd as gq
    c = s["case"]
    if c["op"] == "quantize":
        # the codes, their scales and the values they stand for (the forward
        # value of quantisation-aware training), in one launch
        blocks, scales, values = gq.gq_mxfp4_quantize(s["x"], values=True)
        return {"values": values}
    if c["op"] == "product":
        x = gq.gq_mxfp4_quantize(s["x"])
        if c["rows"] <= 8:
            if c["unit"]:
                y = gq.gq_mxfp4_grouped_gemv_fp4_swiglu(x, s["blocks"], s["scales"], s["ids"])
            else:
                y = gq.gq_mxfp4_grouped_gemv_fp4(x, s["blocks"], s["scales"], s["ids"],
                                                 pair_scale=s["weights"])
            return {"y": y}
        route = gq.gq_route_sort(s["ids"], c["E"])
        if c["unit"]:
            y = gq.gq_mxfp4_grouped_gemm_fp4_swiglu(x, s["blocks"], s["scales"], route)
        else:
            y = gq.gq_mxfp4_grouped_gemm_fp4(x, s["blocks"], s["scales"], route,
                                             pair_scale=s["weights"])
        return {"y": y}
    if c["op"] == "layer":
        return {"y": gq.gq_moe_decode(s["layer"], s["x"])}
    ids, weights = gq.gq_moe_topk(s["logits"], c["topk"], renormalize=c["renorm"])
    got = {"ids": ids, "weights": weights}
    if c["train"]:
        got["d_logits"] = gq.gq_moe_topk_backward(s["d_weights"], s["logits"], ids,
                                                  renormalize=c["renorm"])
    return got


# ---- what a pass cannot do without ---------------------------------------------------
def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["rows"] * c["K"]
        # read once; codes, scales and the bf16 values written once
        return {"bytes": n * (2 + 0.5 + 1 / 32 + (4 if c["dtype"] == "f32" else 2)),
                "flops": 4 * n}
    if c["op"] == "product":
        pairs = c["rows"] * c["topk"]
        used = min(c["E"], pairs) if c["rows"] > 1 else c["topk"]
        out = c["N"] // 2 if c["unit"] else c["N"]
        return {"bytes": c["rows"] * c["K"] * 2 + used * c["N"] * c["K"] * (0.5 + 1 / 32)
                + pairs * out * 2, "flops": 2 * pairs * c["N"] * c["K"]}
    if c["op"] == "layer":
        # experts that rows * topk draws out of E are expected to touch
        E, pairs = c["E"], c["rows"] * c["topk"]
        used = E * (1 - (1 - c["topk"] / E) ** c["rows"])
        per = 0.5 + (4 / 64 if c["fmt"] == "nf4" else 1 / 32)
        return {"bytes": used * 3 * c["I"] * c["H"] * per + E * c["H"] * 2
                + c["rows"] * c["H"] * 4,
                "flops": 2 * pairs * 3 * c["I"] * c["H"] + 2 * c["rows"] * E * c["H"]}
    size = 4 if c["dtype"] == "f32" else 2
    n, k = c["rows"] * c["E"], c["rows"] * c["topk"]
    b = n * size + k * 8
    if c["train"]:
        b += n * size * 2 + k * 8
    return {"bytes": b, "flops": 4 * n * (2 if c["train"] else 1)}


# ---- from the definitions, in 64 bits ----------------------------------------------------
def _q64(x):
    """The nearest e2m1 value by distance, an even code where two are equally near."""
    b = x.double().reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(dim=-1)
    e = torch.where(amax > 0, torch.frexp(torch.where(amax > 0, amax, 1.0)).exponent - 3, -127)
    scale = torch.exp2(e.clamp(-127, 127).double()).unsqueeze(-1)
    v = (b.abs() / scale).clamp(max=6.0)
    order = [0, 2, 4, 6, 1, 3, 5, 7]                       # even codes first
    best = torch.full_like(v, math.inf)
    near = torch.zeros_like(v)
    for code in order:
        d = (v - E2M1[code]).abs()
        near = torch.where(d < best, E2M1[code], near)
        best = torch.minimum(best, d)
    return (torch.copysign(near, b) * scale).reshape(x.shape)


def _w64(fmt, bank, e):
    a, b = bank[0][e], bank[1][e]
    n = a.shape[0]
    v = torch.empty((n, a[0].numel() * 2), dtype=torch.float64, device=a.device)
    a = a.reshape(n, -1).long()
    if fmt == "nf4":
        t = torch.tensor(NF4_BITS).to(torch.int32).view(torch.float32).double().to(a.device)
        v[:, 0::2], v[:, 1::2] = t[a // 16], t[a % 16]
        # a weight is held to be the float32 product of value and absmax
        return (v.float() * b.float().repeat_interleave(64, dim=1)).double()
    t = torch.tensor(E2M1 + [-m for m in E2M1], dtype=torch.float64, device=a.device)
    v[:, 0::2], v[:, 1::2] = t[a % 16], t[a // 16]
    return v * torch.exp2(b.double() - 127).repeat_interleave(32, dim=1)


def _unit64(fmt, h):
    half = h.shape[-1] // 2
    if fmt == "nf4":
        return h[..., :half] * torch.sigmoid(h[..., :half]) * h[..., half:]
    gate = torch.minimum(h[..., 0::2], h.new_tensor(OSS_LIMIT))
    up = torch.clip(h[..., 1::2], -OSS_LIMIT, OSS_LIMIT)
    return gate * torch.sigmoid(OSS_ALPHA * gate) * (up + 1)


def _route64(z, topk, renorm):
    """topk times the largest logit that is left, the first of equal ones."""
    z = z.double()
    left, ids = z.clone(), []
    for _ in range(topk):
        at = (left == left.amax(dim=1, keepdim=True)).to(torch.int8).argmax(dim=1, keepdim=True)
        dead = left.amax(dim=1, keepdim=True) == -math.inf
        ids.append(torch.where(dead, -1, at))
        left = left.scatter(1, at, -math.inf)
    ids = torch.cat(ids, dim=1)
    live = ids >= 0
    chosen = torch.where(live, z.gather(1, ids.clamp(min=0)), -math.inf)
    some = live[:, :1]
    over = chosen if renorm else z
    norm = torch.logsumexp(torch.where(some, over, 0.0), dim=1, keepdim=True)
    return ids, torch.where(live, torch.exp(chosen - norm), 0.0)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    c = case
    if c["op"] == "quantize":
        return {"values": _q64(s["x"])}
    if c["op"] == "product":
        x = _q64(s["x"])
        flat = s["ids"].reshape(-1)
        out = c["N"] // 2 if c["unit"] else c["N"]
        y = torch.zeros((flat.numel(), out), dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            at = (flat == e).nonzero().reshape(-1)
            if at.numel():
                h = x[at // c["topk"]] @ _w64("mxfp4", (s["blocks"], s["scales"]), e).t()
                y[at] = _unit64("mxfp4", h) if c["unit"] else h
        if s["weights"] is not None:
            y *= s["weights"].double()[:, None]
        return {"y": y}
    if c["op"] == "layer":
        x = s["x"].double()
        z = torch.stack([(s["router"].double() * r).sum(dim=1) for r in x])
        if c["bias"]:
            z = z + s["router_bias"].double()
        ids, w = _route64(z, c["topk"], c["renorm"])
        y = torch.zeros((c["rows"], c["H"]), dtype=torch.float64, device=DEV)
        for t, row in enumerate(ids.tolist()):
            for k, e in enumerate(row):
                h = _w64(c["fmt"], s["gate_up"], e) @ x[t]
                if c["bias"]:
                    h = h + s["gate_up_bias"][e].double()
                o = _w64(c["fmt"], s["down"], e) @ _unit64(c["fmt"], h)
                if c["bias"]:
                    o = o + s["down_bias"][e].double()
                y[t] += w[t, k] * o
        return {"y": y}
    ids, w = _route64(s["logits"], c["topk"], c["renorm"])
    got = {"ids": None, "weights": w}
    if c["train"]:
        # the Jacobian of the softmax, row by row of its outputs
        d = s["d_weights"].double()
        z = s["logits"].double()
        some = (z > -math.inf).any(dim=1, keepdim=True)
        if c["renorm"]:
            keep = torch.zeros_like(z).scatter_add(1, ids.clamp(min=0), (ids >= 0).double()) > 0
            z = torch.where(keep, z, -math.inf)
        p = torch.where(some, torch.softmax(torch.where(some, z, 0.0), dim=1), 0.0)
        up = torch.zeros_like(z).scatter_add(1, ids.clamp(min=0), torch.where(ids >= 0, d, 0.0))
        got["d_logits"] = p * up - p * (p * up).sum(dim=1, keepdim=True)
    return got
