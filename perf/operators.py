"""The 8-bit expert layer's operators: the cases that are measured, their inputs and their plain forms.

Formulas. A block is 128 consecutive values of a row; weights have blocks of 128 x 128.
 - scale of a block: the least power of two s with max|v| <= 448 s over the block's finite values v (at least 2^-126);
   q = v / s rounded to e4m3, to nearest, ties to even; a value that is not finite is NaN.
 - norm: r = x + residual, rounded to the type of x; rstd = 1 / sqrt(mean(r^2) + eps); y = r rstd weight, handed on in
   the type of x, in 8 bits with scales, or both (each rounded from the unrounded y).
 - its gradient: g = dy weight; dx = rstd (g - r rstd^2 mean(g r)) + dresidual; dweight = sum over rows of dy r rstd.
 - grouped product: out[s, :] = a[row(s), :] W_e^T for the rows s of expert e, both operands in 8 bits with scales;
   weights are [E, out, in].
 - expert layer: h = x W_up_e^T; a = silu(gate) up, put in 8 bits per block of a row; y = a W_down_e^T;
   out[t] = sum over the token's slots of topk_weight y.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
TOP = 448.0  # the largest e4m3 value
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def cdiv(a, b):
    return -(-a // b)


def listed():
    return [
        # one decoded token ahead of the 8-bit experts: latency alone
        {"name": "norm 1 token", "op": "norm", "N": 1, "H": 7168, "dtype": "bf16", "residual": True, "y": True, "q": True, "scale": "e8m0"},
        # the default workload's tokens: the router reads y, the experts q
        {"name": "norm 16384 x 2048", "op": "norm", "N": 16384, "H": 2048, "dtype": "bf16", "residual": True, "y": True, "q": True, "scale": "e8m0"},
        # a ragged width whose last block is partial, 8 bits only, no residual stream
        {"name": "norm 5003 x 1000", "op": "norm", "N": 5003, "H": 1000, "dtype": "bf16", "residual": False, "y": False, "q": True, "scale": "e8m0"},
        # the norm's gradient on the default workload
        {"name": "norm grad 16384 x 2048", "op": "norm_grad", "N": 16384, "H": 2048, "dtype": "bf16", "residual": True},
        # a short ragged batch in 32 bits, with no residual stream behind it
        {"name": "norm grad 333 x 5000 fp32", "op": "norm_grad", "N": 333, "H": 5000, "dtype": "fp32", "residual": False},
        # the up projections of the default workload's experts, after a step of training
        {"name": "weights 32 x 2048 x 1024", "op": "quantize_weights", "E": 32, "K": 2048, "C": 1024, "dtype": "bf16", "scale": "e8m0"},
        # received rows that come in 16 bits; the scales in 32 bits, as a dispatch sends them
        {"name": "rows 8192 x 7168", "op": "quantize_rows", "N": 8192, "H": 7168, "dtype": "bf16", "scale": "fp32"},
        # eight decoded tokens: the weights' bytes are the time
        {"name": "experts 8 tokens", "op": "experts", "N": 8, "H": 7168, "I": 2048, "E": 32, "K": 8, "drop": 0.5, "skew": 0.0, "scale": "e8m0", "layout": "interleaved", "save": False},
        # the default workload: an eighth of 256 experts, h kept for the backward
        {"name": "experts 16384 tokens", "op": "experts", "N": 16384, "H": 2048, "I": 512, "E": 32, "K": 8, "drop": 0.93, "skew": 0.0, "scale": "e8m0", "layout": "interleaved", "save": True},
        # uneven experts and a checkpoint's form: scales in 32 bits, gates and ups one after the other
        {"name": "experts 8192 tokens uneven", "op": "experts", "N": 8192, "H": 7168, "I": 2048, "E": 32, "K": 8, "drop": 0.91, "skew": 1.1, "scale": "fp32", "layout": "concat", "save": False},
        # a small batch of odd sizes through one product of an expert
        {"name": "product 100 tokens odd", "op": "product", "N": 100, "C": 1040, "D": 592, "E": 12, "K": 3, "drop": 0.1, "skew": 0.5, "scale": "fp32"},
        # the largest product: long prompts
        {"name": "product 65536 tokens", "op": "product", "N": 65536, "C": 4096, "D": 4096, "E": 64, "K": 6, "drop": 0.5, "skew": 0.0, "scale": "e8m0"},
    ]


def spread(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], {"bytes": 0, "flops": 0})
        for k in m:
            m[k] = max(m[k], w[k])
    while True:
        op = rng.choice(("norm", "norm_grad", "quantize_weights", "quantize_rows", "experts", "experts", "product"))
        scale = rng.choice(("e8m0", "fp32"))
        if op in ("norm", "norm_grad", "quantize_rows"):
            c = {"op": op, "N": spread(rng, 1, 32768), "H": spread(rng, 64, 8192, 8), "dtype": rng.choice(("bf16", "bf16", "fp32"))}
            if op == "norm":
                y, q = rng.choice(((True, False), (False, True), (True, True)))
                c.update(residual=rng.random() < 0.6, y=y, q=q, scale="e8m0")
            elif op == "norm_grad":
                c.update(residual=rng.random() < 0.6)
            else:
                c.update(scale=scale)
        elif op == "quantize_weights":
            c = {"op": op, "E": spread(rng, 1, 64), "K": spread(rng, 64, 7168, 16), "C": spread(rng, 64, 4096, 16), "dtype": rng.choice(("bf16", "bf16", "fp32")), "scale": scale}
        else:
            E = spread(rng, 1, 64)
            c = {"op": op, "N": spread(rng, 1, 16384), "E": E, "K": min(E, rng.randint(1, 8)), "drop": rng.choice((0.0, 0.1, 0.5, 0.8)), "skew": rng.choice((0.0, 0.0, 0.5, 1.1)), "scale": scale}
            if op == "experts":
                c.update(H=spread(rng, 128, 7168, 16), I=spread(rng, 64, 2048, 16), layout=rng.choice(("interleaved", "concat")), save=rng.random() < 0.4)
            else:
                c.update(C=spread(rng, 64, 7168, 16), D=spread(rng, 64, 7168, 16))
        w = work(c)
        if all(w[k] <= most[op][k] for k in w) and w["bytes"] > 0:
            return c


# ---- inputs ---------------------------------------------------------------------------------------------------------


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def stream_rows(g, N, H, dtype):
    """Activations: some channels are far larger than the others, and rows differ in size."""
    col = torch.exp(0.5 * torch.randn(H, generator=g, device=DEV))
    col[torch.rand(H, generator=g, device=DEV) < 0.004] *= 20.0
    row = torch.exp(0.3 * torch.randn(N, 1, generator=g, device=DEV))
    return (torch.randn(N, H, generator=g, device=DEV) * col * row).to(dtype)


def power_scale(amax):
    """The least power of two s with amax <= 448 s, at least 2^-126, from the exponent's bits."""
    bits = amax.float().contiguous().view(torch.int32)
    e = ((bits + 0x1FFFFF) >> 23) - 8  # the mantissa of 448 is 1.75
    return e.clamp(min=1).bitwise_left_shift(23).view(torch.float32)


def by_blocks(v):
    """[..., L] -> [..., ceil(L/128), 128], with zeros behind the end."""
    L = v.shape[-1]
    n = cdiv(L, BLOCK)
    if n * BLOCK != L:
        v = torch.nn.functional.pad(v, (0, n * BLOCK - L))
    return v.unflatten(-1, (n, BLOCK))


def to_8_bits(v, s):
    return torch.where(torch.isfinite(v), v / s, float("nan")).to(torch.float8_e4m3fn)


def quantize_rows(v):
    """fp32 [N, L] -> e4m3 [N, L], fp32 power-of-two scales [N, ceil(L/128)]."""
    b = by_blocks(v)
    s = power_scale(torch.where(torch.isfinite(b), b.abs(), 0.0).amax(-1))
    return to_8_bits(b, s[..., None]).view(torch.uint8).flatten(-2)[..., : v.shape[-1]].contiguous().view(torch.float8_e4m3fn), s


def quantize_blocks(w, power):
    """fp32 [E, R, C] -> e4m3 [E, R, C], fp32 scales [E, ceil(R/128), ceil(C/128)], powers of two or not."""
    E, R, C = w.shape
    nr, nc = cdiv(R, BLOCK), cdiv(C, BLOCK)
    p = torch.nn.functional.pad(w, (0, nc * BLOCK - C, 0, nr * BLOCK - R)) if R % BLOCK or C % BLOCK else w
    b = p.view(E, nr, BLOCK, nc, BLOCK)
    amax = torch.where(torch.isfinite(b), b.abs(), 0.0).amax((2, 4))
    s = power_scale(amax) if power else (amax / TOP).clamp(min=2.0**-126)
    q = to_8_bits(b, s[:, :, None, :, None]).view(torch.uint8).reshape(E, nr * BLOCK, nc * BLOCK)[:, :R, :C]
    return q.contiguous().view(torch.float8_e4m3fn), s


def as_scale(s, kind):
    """Scales as they are kept: fp32, or the exponent's byte."""
    return s.contiguous() if kind == "fp32" else (s.contiguous().view(torch.int32) >> 23).to(torch.uint8).view(torch.float8_e8m0fnu)


def weights(g, E, R, C, kind):
    """A checkpoint's expert weights [E, R, C] in 8 bits: made once, kept by the program."""
    q, s = [], []
    for _ in range(E):
        w = torch.randn(1, R, C, generator=g, device=DEV) * 0.02
        a, b = quantize_blocks(w, kind == "e8m0")
        q.append(a.view(torch.uint8))
        s.append(b)
    return torch.cat(q).view(torch.float8_e4m3fn), as_scale(torch.cat(s), kind)


def rows_8_bits(g, N, H, kind):
    """Received rows in 8 bits; scales in 32 bits need not be powers of two."""
    v = stream_rows(g, N, H, torch.float32)
    if kind == "e8m0":
        q, s = quantize_rows(v)
    else:
        b = by_blocks(v)
        s = (b.abs().amax(-1) / TOP).clamp(min=2.0**-126)
        q = to_8_bits(b, s[..., None]).view(torch.uint8).flatten(-2)[..., :H].contiguous().view(torch.float8_e4m3fn)
    return q, as_scale(s, kind)


def dropped(N, K, drop):
    """Slots that are -1: a share of those but one of every row."""
    return int(round(drop * N * (K - 1)))


def routing(g, N, E, K, drop, skew):
    """topk_idx [N, K] with -1 for slots of other ranks, every row with one at least; topk_weights; rows per expert."""
    pop = -skew * torch.log(1.0 + torch.randperm(E, generator=g, device=DEV).float())
    u = torch.rand(N, E, generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)
    idx = torch.topk(pop - torch.log(-torch.log(u)), K, dim=1).indices.to(torch.int32)
    first = torch.rand(N, K, generator=g, device=DEV)
    first.scatter_(1, torch.randint(0, K, (N, 1), generator=g, device=DEV), 2.0)
    gone = torch.zeros(N * K, dtype=torch.bool, device=DEV)
    gone[torch.topk(first.flatten(), dropped(N, K, drop), largest=False).indices] = True  # as many whatever the seed
    gone = gone.view(N, K)
    w = torch.softmax(torch.randn(N, K, generator=g, device=DEV).masked_fill(gone, -math.inf), 1)
    idx = idx.masked_fill(gone, -1)
    counts = torch.bincount((idx + 1).flatten().long(), minlength=E + 1)[1:]
    return idx.contiguous(), w.contiguous(), [int(c) for c in counts.cpu()]


def prepare(case, seed):
    g = generator(seed)
    c, s = case, {"case": case}
    if c["op"] in ("norm", "norm_grad"):
        N, H, dt = c["N"], c["H"], DTYPES[c["dtype"]]
        s["x"] = stream_rows(g, N, H, dt)
        s["weight"] = (1.0 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(dt)
        if c["op"] == "norm":
            s["residual"] = normal(g, (N, H), dt, 4.0) if c["residual"] else None
        else:
            s["rstd"] = 1.0 / torch.sqrt(s["x"].float().square().mean(1) + EPS)  # kept by the forward, x as its r
            s["dy"] = normal(g, (N, H), dt)
            s["dresidual"] = normal(g, (N, H), dt) if c["residual"] else None
    elif c["op"] == "quantize_rows":
        s["x"] = stream_rows(g, c["N"], c["H"], DTYPES[c["dtype"]])
    elif c["op"] == "quantize_weights":
        s["w"] = normal(g, (c["E"], c["K"], c["C"]), DTYPES[c["dtype"]], 0.02)
    else:
        width = c["H"] if c["op"] == "experts" else c["C"]
        s["idx"], s["topk"], s["counts"] = routing(g, c["N"], c["E"], c["K"], c["drop"], c["skew"])
        s["x"], s["x_scale"] = rows_8_bits(g, c["N"], width, c["scale"])
        if c["op"] == "experts":
            s["up"], s["up_scale"] = weights(g, c["E"], 2 * c["I"], c["H"], c["scale"])
            s["down"], s["down_scale"] = weights(g, c["E"], c["H"], c["I"], c["scale"])
        else:
            s["w"], s["w_scale"] = weights(g, c["E"], c["D"], c["C"], c["scale"])
    return s


# ---- one pass -------------------------------------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm": own_norm, "norm_grad": own_norm_grad, "quantize_rows": own_quantize, "quantize_weights": own_quantize,
                "experts": own_experts, "product": own_product}[op](s)
    return {"norm": plain_norm, "norm_grad": plain_norm_grad, "quantize_rows": plain_quantize, "quantize_weights": plain_quantize,
            "experts": plain_experts, "product": plain_product}[op](s)


def plain_norm(s):
    c, x = s["case"], s["x"]
    out = {}
    r = x
    if s["residual"] is not None:
        r = out["r"] = (x.float() + s["residual"].float()).to(x.dtype)
    v = r.float()
    out["rstd"] = 1.0 / torch.sqrt(v.square().mean(1) + EPS)
    y = v * out["rstd"][:, None] * s["weight"].float()
    if c["y"]:
        out["y"] = y.to(x.dtype)
    if c["q"]:
        out["q"], scale = quantize_rows(y)
        out["scale"] = as_scale(scale, c["scale"])
    return out


def plain_norm_grad(s):
    r, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    gr = dy * s["weight"].float()
    dx = rstd * (gr - r * (rstd * rstd * (gr * r).mean(1, keepdim=True)))
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * (r * rstd)).sum(0).to(s["x"].dtype)}


def plain_quantize(s):
    c = s["case"]
    if c["op"] == "quantize_rows":
        q, scale = quantize_rows(s["x"].float())
    else:
        q, scale = quantize_blocks(s["w"].float().transpose(1, 2).contiguous(), True)
    return {"q": q, "scale": as_scale(scale, c["scale"])}


def wide_rows(q, s, idx):
    """fp32 values of rows idx of an 8-bit tensor with scales per block of a row."""
    v = q.view(torch.uint8)[idx].view(torch.float8_e4m3fn).float()
    sc = s.float()[idx] if s.dtype == torch.float32 else s.view(torch.uint8)[idx].view(torch.float8_e8m0fnu).float()
    return v * sc.repeat_interleave(BLOCK, 1)[:, : v.shape[1]]


def wide_weights(q, s, e):
    """fp32 values of expert e's weights."""
    R, C = q.shape[1:]
    return q[e].float() * s[e].float().repeat_interleave(BLOCK, 0)[:R].repeat_interleave(BLOCK, 1)[:, :C]


def sorted_slots(s):
    """The valid slots by expert, and each one's row."""
    c = s["case"]
    key = torch.where(s["idx"] < 0, c["E"], s["idx"]).flatten()
    slots = torch.sort(key, stable=True).indices[: sum(s["counts"])]
    return slots, slots // c["K"]


def segments(counts):
    at, found = 0, []
    for e, n in enumerate(counts):
        if n:
            found.append((e, at, at + n))
        at += n
    return found


def plain_product(s):
    c = s["case"]
    _, rows = sorted_slots(s)
    out = torch.empty(len(rows), c["D"], device=DEV)
    for e, a, b in segments(s["counts"]):
        out[a:b] = wide_rows(s["x"], s["x_scale"], rows[a:b]) @ wide_weights(s["w"], s["w_scale"], e).t()
    return out.to(torch.bfloat16)


def plain_experts(s):
    c = s["case"]
    N, H, I, K = c["N"], c["H"], c["I"], c["K"]
    slots, rows = sorted_slots(s)
    y = torch.zeros(N * K, H, device=DEV)
    kept = torch.empty(len(rows), 2 * I, device=DEV, dtype=torch.bfloat16) if c["save"] else None
    wt = s["topk"].flatten()
    for e, a, b in segments(s["counts"]):
        h = wide_rows(s["x"], s["x_scale"], rows[a:b]) @ wide_weights(s["up"], s["up_scale"], e).t()
        gate, up = (h[:, :I], h[:, I:]) if c["layout"] == "concat" else (h[:, 0::2], h[:, 1::2])
        if c["save"]:
            kept[a:b] = torch.stack((gate, up), 2).flatten(1).to(torch.bfloat16)
        q, sc = quantize_rows(gate / (1.0 + torch.exp(-gate)) * up)
        v = q.float() * sc.repeat_interleave(BLOCK, 1)[:, :I]
        y[slots[a:b]] = (v @ wide_weights(s["down"], s["down_scale"], e).t()) * wt[slots[a:b], None]
    out = {"out": y.view(N, K, H).sum(1).to(torch.bfloat16)}
    if c["save"]:
        out["h"] = kept
    return out


# ---- the framework's calls ------------------------------------------------------------------------------------------


def scale_like(c, *shape):
    return torch.empty(shape, device=DEV, dtype=torch.float32 if c["scale"] == "fp32" else torch.float8_e8m0fnu)


def own_norm(s):
    import token_routing_grouped_amd as moe

    c, x = s["case"], s["x"]
    N, H = x.shape
    out = {"rstd": torch.empty(N, device=DEV)}
    if s["residual"] is not None:
        out["r"] = torch.empty_like(x)
    if c["y"]:
        out["y"] = torch.empty_like(x)
    if c["q"]:
        out["q"] = torch.empty(N, H, device=DEV, dtype=torch.float8_e4m3fn)
        out["scale"] = scale_like(c, N, cdiv(H, BLOCK))
    moe.moe_rmsnorm_forward(x, s["weight"], EPS, residual=s["residual"], residual_out=out.get("r"), y=out.get("y"),
                            q=out.get("q"), scale=out.get("scale"), rstd=out["rstd"])
    return out


def own_norm_grad(s):
    import token_routing_grouped_amd as moe

    out = {"dx": torch.empty_like(s["x"]), "dweight": torch.empty_like(s["weight"])}
    moe.moe_rmsnorm_backward(s["dy"], s["x"], s["weight"], s["rstd"], out["dx"], out["dweight"], dresidual=s["dresidual"])
    return out


def own_quantize(s):
    import token_routing_grouped_amd as moe

    c = s["case"]
    if c["op"] == "quantize_rows":
        q = torch.empty(c["N"], c["H"], device=DEV, dtype=torch.float8_e4m3fn)
        scale = scale_like(c, c["N"], cdiv(c["H"], BLOCK))
        moe.moe_quantize_rows(s["x"], q, scale)
    else:
        q = torch.empty(c["E"], c["C"], c["K"], device=DEV, dtype=torch.float8_e4m3fn)
        scale = scale_like(c, c["E"], cdiv(c["C"], BLOCK), cdiv(c["K"], BLOCK))
        moe.moe_quantize_weights(s["w"], q, scale)
    return {"q": q, "scale": scale}


def own_metadata(s):
    """The program's metadata object, built anew for each batch's routing."""
    import token_routing_grouped_amd as moe

    c = s["case"]
    if "meta" not in s:
        s["meta"] = moe.Metadata(c["N"], c["K"], c["E"], sum(s["counts"]), device=torch.device(DEV, torch.cuda.current_device()))
    moe.moe_build_metadata(s["idx"], s["topk"], s["meta"])
    return s["meta"]


def own_product(s):
    import token_routing_grouped_amd as moe

    c, meta = s["case"], own_metadata(s)
    out = torch.empty(meta.capacity, c["D"], device=DEV, dtype=torch.bfloat16)
    moe.moe_grouped_gemm_fp8(meta, s["x"], s["x_scale"], s["w"], s["w_scale"], out, gather=True)
    return out


def own_experts(s):
    import token_routing_grouped_amd as moe

    c, meta = s["case"], own_metadata(s)
    out = {"out": torch.empty(c["N"], c["H"], device=DEV, dtype=torch.bfloat16)}
    if c["save"]:
        out["h"] = torch.empty(meta.capacity, 2 * c["I"], device=DEV, dtype=torch.bfloat16)
    layout = moe.MOE_GATEUP_CONCAT if c["layout"] == "concat" else moe.MOE_GATEUP_INTERLEAVED
    moe.moe_expert_forward_fp8(meta, s["x"], s["x_scale"], s["up"], s["up_scale"], s["down"], s["down_scale"], out["out"],
                               h_save=out.get("h"), layout=layout)
    return out


# ---- what a pass cannot do without ----------------------------------------------------------------------------------


def pairs_of(c):
    """The (row, expert) pairs of a routed case, and how many experts are expected to have rows."""
    pairs = c["N"] * c["K"] - dropped(c["N"], c["K"], c["drop"])
    return pairs, c["E"] * (1.0 - (1.0 - 1.0 / c["E"]) ** pairs)


def work(case):
    c = case
    es = {"bf16": 2, "fp32": 4}
    sb = {"e8m0": 1, "fp32": 4}.get(c.get("scale"), 0)
    if c["op"] in ("norm", "norm_grad", "quantize_rows"):
        n, e = c["N"] * c["H"], es[c["dtype"]]
        sc = c["N"] * cdiv(c["H"], BLOCK) * sb
        if c["op"] == "norm":
            b = n * e * (3 if c["residual"] else 1) + (n * e if c["y"] else 0) + (n + sc if c["q"] else 0) + c["H"] * e + 4 * c["N"]
            return {"bytes": b, "flops": 8 * n}
        if c["op"] == "norm_grad":
            return {"bytes": n * e * (4 if c["residual"] else 3) + 2 * c["H"] * e + 4 * c["N"], "flops": 10 * n}
        return {"bytes": n * (e + 1) + sc, "flops": 3 * n}
    if c["op"] == "quantize_weights":
        n = c["E"] * c["K"] * c["C"]
        return {"bytes": n * (es[c["dtype"]] + 1) + c["E"] * cdiv(c["K"], BLOCK) * cdiv(c["C"], BLOCK) * sb, "flops": 3 * n}
    P, live = pairs_of(c)
    routed = c["N"] * c["K"] * 8
    if c["op"] == "product":
        b = c["N"] * c["C"] + live * c["C"] * c["D"] + P * c["D"] * 2 + routed
        return {"bytes": int(b), "flops": int(2 * P * c["C"] * c["D"])}
    b = c["N"] * c["H"] + live * 3 * c["H"] * c["I"] + c["N"] * c["H"] * 2 + (P * c["I"] * 4 if c["save"] else 0) + routed
    return {"bytes": int(b), "flops": int(6 * P * c["H"] * c["I"])}


# ---- from the definitions, in 64 bits -------------------------------------------------------------------------------


def two_to(k):
    """2^k in 64 bits, from its exponent's bits."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def exact_scale(amax):
    m, e = torch.frexp(amax / 448.0)  # amax / 448 = m 2^e, 1/2 <= m < 1
    k = torch.where(m > 0.5, e, e - 1)
    return two_to(torch.where(amax > 0, k, -126).clamp(min=-126))


def exact_e4m3(v):
    """Nearest value with three mantissa bits, ties to even; steps of 2^-9 below 2^-6."""
    e = (torch.frexp(v)[1] - 1).clamp(min=-6)
    step = two_to(e - 3)
    return torch.round(v / step) * step


def exact_rows(v):
    """(quotients on e4m3, scales, the values they stand for) of fp64 [N, L]."""
    q, s = torch.empty_like(v), []
    for k in range(0, v.shape[1], BLOCK):
        part = v[:, k : k + BLOCK]
        one = exact_scale(part.abs().amax(1))
        q[:, k : k + BLOCK] = exact_e4m3(part / one[:, None])
        s.append(one)
    s = torch.stack(s, 1)
    return q, s, q * s.repeat_interleave(BLOCK, 1)[:, : v.shape[1]]


def exact_routed(s):
    """[(expert, rows, slot numbers)] in order of the experts, from the routing on the host."""
    idx, found = s["idx"].cpu().flatten(), []
    K = s["case"]["K"]
    for e in range(s["case"]["E"]):
        at = torch.nonzero(idx == e).flatten().to(DEV)
        if len(at):
            found.append((e, at // K, at))
    return found


def exact_weight(q, s, e):
    v = q[e].double()
    sc = s[e].double()
    i = torch.arange(v.shape[0], device=DEV) // BLOCK
    j = torch.arange(v.shape[1], device=DEV) // BLOCK
    return v * sc[i][:, j]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        r = s["x"].double()
        out = {}
        if s["residual"] is not None:
            r = out["r"] = (r + s["residual"].double()).to(s["x"].dtype).double()
        out["rstd"] = (r.pow(2).sum(1) / c["H"] + EPS).pow(-0.5)
        y = r * s["weight"].double() * out["rstd"][:, None]
        if c["y"]:
            out["y"] = y
        if c["q"]:
            out["q"], out["scale"], _ = exact_rows(y)
        return out
    if c["op"] == "norm_grad":
        r, dy, w, t = s["x"].double(), s["dy"].double(), s["weight"].double(), s["rstd"].double()[:, None]
        n = r * t  # the normalized rows
        gn = dy * w
        dx = t * (gn - n * (gn * n).sum(1, keepdim=True) / c["H"])
        if s["dresidual"] is not None:
            dx = dx + s["dresidual"].double()
        return {"dx": dx, "dweight": (dy * n).sum(0)}
    if c["op"] == "quantize_rows":
        q, sc, _ = exact_rows(s["x"].double())
        return {"q": q, "scale": sc}
    if c["op"] == "quantize_weights":
        w = s["w"].double().transpose(1, 2)
        q = torch.empty(w.shape, dtype=torch.float64, device=DEV)
        sc = torch.empty(c["E"], cdiv(c["C"], BLOCK), cdiv(c["K"], BLOCK), dtype=torch.float64, device=DEV)
        for i in range(sc.shape[1]):
            for j in range(sc.shape[2]):
                at = (slice(None), slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
                sc[:, i, j] = exact_scale(w[at].abs().amax((1, 2)))
                q[at] = exact_e4m3(w[at] / sc[:, i, j][:, None, None])
        return {"q": q, "scale": sc}
    x = s["x"].double() * s["x_scale"].double().repeat_interleave(BLOCK, 1)[:, : s["x"].shape[1]]
    if c["op"] == "product":
        return torch.cat([x[rows] @ exact_weight(s["w"], s["w_scale"], e).t() for e, rows, _ in exact_routed(s)])
    I, out, kept = c["I"], torch.zeros(c["N"], c["H"], dtype=torch.float64, device=DEV), []
    for e, rows, at in exact_routed(s):
        h = x[rows] @ exact_weight(s["up"], s["up_scale"], e).t()
        j = torch.arange(I, device=DEV)
        gate, up = (h[:, j], h[:, I + j]) if c["layout"] == "concat" else (h[:, 2 * j], h[:, 2 * j + 1])
        kept.append(torch.stack((gate, up), 2).reshape(len(rows), 2 * I))
        a = exact_rows(gate * torch.sigmoid(gate) * up)[2]
        out.index_add_(0, rows, (a @ exact_weight(s["down"], s["down_scale"], e).t()) * s["topk"].double().flatten()[at][:, None])
    return {"out": out, "h": torch.cat(kept)} if c["save"] else {"out": out}
