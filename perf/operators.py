"""Cases and plain forms of the operators around the quantized products of a decoder layer.

Four operators are measured: the root-mean-square norm with the residual's
addition that writes Q8_1 activations, reading Q8_1 activations back, the
routing of tokens to experts, and the matrix-vector product of 4-bit weights
with group scales.  Each has a plain form here, made of elementary torch
operations in 32 bits, and an exact form in 64 bits.

Where ``own`` is true, ``run`` calls the library instead.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2, "": 0}

# The largest sizes that draw() gives: those of the largest listed case of each operator.
MOST_NORM, MOST_READ, MOST_ROUTE, MOST_MATVEC = 16384 * 8192, 8192 * 11008, 32768 * 384, 28672 * 8192


def listed():
    return [
        # One decoded token between two products: the fp32 output of a matvec joins a bf16 residual stream.
        {"name": "norm 1x4096", "op": "norm", "T": 1, "K": 4096, "x": "f32", "res": "bf16", "w": "bf16", "y": "",
         "offset": 0.0, "eps": 1e-5},
        # A small ragged batch, first norm of a model (no residual yet), 16-bit copy kept, weights stored as w - 1.
        {"name": "norm 37x2080", "op": "norm", "T": 37, "K": 2080, "x": "f16", "res": "", "w": "f32", "y": "f16",
         "offset": 1.0, "eps": 1e-6},
        # The hidden rows of a 512-token routed FFN layer: Q8_1 for the experts, bf16 for the router's projection.
        {"name": "norm 512x2048", "op": "norm", "T": 512, "K": 2048, "x": "f32", "res": "f32", "w": "f32", "y": "bf16",
         "offset": 0.0, "eps": 1e-6},
        # A long prompt of a wide model.
        {"name": "norm 16384x8192", "op": "norm", "T": 16384, "K": 8192, "x": "bf16", "res": "bf16", "w": "bf16",
         "y": "", "offset": 0.0, "eps": 1e-5},
        # Q8_1 rows read back for a consumer that is not quantized: a few tokens, and the FFN rows of a long prompt.
        {"name": "read 5x4096", "op": "read", "T": 5, "K": 4096, "y": "f32"},
        {"name": "read 8192x11008", "op": "read", "T": 8192, "K": 11008, "y": "bf16"},
        # One decoded token of the 128-expert layer, raw softmax probabilities.
        {"name": "route 1x128", "op": "route", "T": 1, "E": 128, "top_k": 8, "x": "f32", "scoring": "softmax",
         "bias": False, "groups": 1, "keep": 1, "group_score": "max", "renorm": False, "scale": 1.0, "masked": False},
        # A prompt through sigmoid scores with a balancing bias, half of the expert groups kept, renormalised.
        {"name": "route 4099x256", "op": "route", "T": 4099, "E": 256, "top_k": 8, "x": "bf16", "scoring": "sigmoid",
         "bias": True, "groups": 8, "keep": 4, "group_score": "top2", "renorm": True, "scale": 2.0, "masked": False},
        # A long prompt over an expert count that is no power of two, softmax with a bias, some experts masked.
        {"name": "route 32768x384", "op": "route", "T": 32768, "E": 384, "top_k": 6, "x": "f32", "scoring": "softmax",
         "bias": True, "groups": 1, "keep": 1, "group_score": "max", "renorm": True, "scale": 1.0, "masked": True},
        # A small projection of one token, where the launch counts.
        {"name": "matvec 1024x1024 T1", "op": "matvec", "T": 1, "M": 1024, "K": 1024, "group": 64, "scale": "f16",
         "zeros": False},
        # The decode shape of the k-quant matvecs, one token, with zero points.
        {"name": "matvec 4096x11008 T1", "op": "matvec", "T": 1, "M": 4096, "K": 11008, "group": 128, "scale": "f16",
         "zeros": True},
        # A wide gate and up projection for a few tokens at once (several sequences, or drafted tokens), small groups.
        {"name": "matvec 28672x8192 T5", "op": "matvec", "T": 5, "M": 28672, "K": 8192, "group": 32, "scale": "bf16",
         "zeros": False},
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    op = rng.choice(["norm", "norm", "read", "route", "route", "matvec", "matvec"])
    if op in ("norm", "read"):
        K = 32 * spread(1, 512)
        T = spread(1, min(16384, (MOST_NORM if op == "norm" else MOST_READ) // K))
        if op == "read":
            return {"op": op, "T": T, "K": K, "y": rng.choice(list(DTYPES))}
        return {"op": op, "T": T, "K": K, "x": rng.choice(list(DTYPES)), "res": rng.choice(["", *DTYPES]),
                "w": rng.choice(list(DTYPES)), "y": rng.choice(["", *DTYPES]), "offset": rng.choice([0.0, 1.0]),
                "eps": rng.choice([1e-6, 1e-5])}
    if op == "route":
        groups = rng.choice([1, 1, 1, 2, 4, 8])
        per = spread(2, 512 // groups)
        keep = rng.randint(1, groups)
        E = groups * per
        return {"op": op, "T": spread(1, min(32768, MOST_ROUTE // E)), "E": E,
                "top_k": rng.randint(1, min(16, keep * per)), "x": rng.choice(list(DTYPES)),
                "scoring": rng.choice(["softmax", "sigmoid"]), "bias": rng.choice([False, True]), "groups": groups,
                "keep": keep, "group_score": rng.choice(["max", "top2"]), "renorm": rng.choice([False, True]),
                "scale": rng.choice([1.0, 1.5]), "masked": rng.choice([False, False, True])}
    group = rng.choice([32, 64, 128])
    K = group * spread(1, 16384 // group)
    return {"op": op, "T": rng.randint(1, 8), "M": spread(1, min(65536, MOST_MATVEC // K)), "K": K,
            "group": rng.choice([group, group, group, K]), "scale": rng.choice(["f16", "bf16"]),
            "zeros": rng.choice([False, True])}


def work(case):
    c = case
    if c["op"] == "norm":
        # the norm, and reading its Q8_1 rows back: x, the residual in and out, the unquantized copy, 40 bytes of
        # Q8_1 for 32 values written and read, and a 16-bit value each
        each = SIZES[c["x"]] + 2 * SIZES[c["res"]] + SIZES[c["y"]] + 2 * 1.25 + 2
        return {"bytes": c["T"] * c["K"] * each + c["K"] * SIZES[c["w"]], "flops": 12.0 * c["T"] * c["K"]}
    if c["op"] == "read":
        return {"bytes": c["T"] * c["K"] * (1.25 + SIZES[c["y"]]), "flops": 1.0 * c["T"] * c["K"]}
    if c["op"] == "route":
        # a score for each expert, and one comparison of each for each of the chosen
        return {"bytes": c["T"] * (c["E"] * SIZES[c["x"]] + c["top_k"] * 8) + 4 * c["E"] * c["bias"],
                "flops": float(c["T"] * c["E"] * (4 + c["top_k"]))}
    groups = c["K"] // c["group"]
    row = c["K"] / 2 + 2 * groups + (groups + 1) // 2 * c["zeros"]
    return {"bytes": c["M"] * row + c["T"] * (c["K"] * 1.25 + 4 * c["M"]), "flops": 2.0 * c["T"] * c["M"] * c["K"]}


# ---------------------------------------------------------------- inputs


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _q8_1_rows(g, T, K):
    """Q8_1 rows of N(0, 1) activations with 1% outliers: per 32 values an f16 scale, two zero bytes, 32 int8, int32 sum."""
    x = _normal(g, T, K)
    x = torch.where(_uniform(g, T, K) < 0.01, x * 20.0, x).view(T, K // 32, 32)
    d = x.abs().amax(-1, keepdim=True) / 127.0
    q = torch.round(x / d.clamp_min(1e-30)).clamp(-127, 127).to(torch.int8)
    out = torch.zeros(T, K // 32, 40, dtype=torch.uint8, device=DEVICE)
    out[..., 0:2] = d.to(torch.float16).view(torch.uint8)
    out[..., 4:36] = q.view(torch.uint8)
    out[..., 36:40] = q.sum(-1, keepdim=True, dtype=torch.int32).view(torch.uint8)
    return out


def prepare(case, seed):
    c, g = case, torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"case": dict(c)}
    if c["op"] == "norm":
        # a stream with a few channels far larger than the rest, as hidden states have them
        loud = torch.where(_uniform(g, c["K"]) < 0.004, 12.0, 1.0)
        s["x"] = (_normal(g, c["T"], c["K"]) * loud * 0.7).to(DTYPES[c["x"]])
        s["res"] = (_normal(g, c["T"], c["K"]) * loud * 2.0).to(DTYPES[c["res"]]) if c["res"] else None
        s["w"] = (1.0 - c["offset"] + 0.2 * _normal(g, c["K"])).to(DTYPES[c["w"]])
    elif c["op"] == "read":
        s["xq"] = _q8_1_rows(g, c["T"], c["K"])
    elif c["op"] == "route":
        x = _normal(g, c["T"], c["E"]) * 1.5
        if c["masked"]:
            # some experts switched off for everyone, some for single tokens, and now and then a token without any
            x = x.masked_fill(_uniform(g, c["E"]) < 0.1, -math.inf).masked_fill(_uniform(g, c["T"], c["E"]) < 0.05, -math.inf)
            x = x.masked_fill(_uniform(g, c["T"], 1) < 0.02, -math.inf)
        s["logits"] = x.to(DTYPES[c["x"]])
        s["bias"] = 0.05 * _normal(g, c["E"]) if c["bias"] else None
    else:
        M, K, n = c["M"], c["K"], c["K"] // c["group"]
        s["w"] = torch.randint(0, 256, (M, K // 2), generator=g, device=DEVICE, dtype=torch.uint8)
        s["scales"] = (0.01 * (0.5 + _uniform(g, M, n))).to(DTYPES[c["scale"]])
        s["zeros"] = None
        if c["zeros"]:
            # zero points near the middle, as min-max fits of weights have them
            z = torch.randint(5, 11, (M, (n + 1) // 2 * 2), generator=g, device=DEVICE, dtype=torch.uint8)
            s["zeros"] = (z[:, 0::2] | (z[:, 1::2] << 4)).contiguous()
        s["xq"] = _q8_1_rows(g, c["T"], K)
    return s


# ---------------------------------------------------------------- the library's calls


def _run_own(s):
    import quantized_matmul_q8_amd as qmm

    c = s["case"]
    if c["op"] == "norm":
        xq, res, y = qmm.rms_norm_q8_1(s["x"], s["w"], c["eps"], residual=s["res"], weight_offset=c["offset"],
                                       y_dtype=DTYPES[c["y"]] if c["y"] else None)
        return qmm.q8_1_dequantize(xq, torch.float16), res, y
    if c["op"] == "read":
        return qmm.q8_1_dequantize(s["xq"], DTYPES[c["y"]])
    if c["op"] == "route":
        return qmm.moe_router(s["logits"], c["top_k"], scoring=c["scoring"], bias=s["bias"], n_groups=c["groups"],
                              topk_groups=c["keep"], group_score=c["group_score"], renormalize=c["renorm"],
                              scale=c["scale"])
    return qmm.mmvq_q4g(s["w"], s["scales"], s["xq"], zeros=s["zeros"])


# ---------------------------------------------------------------- plain forms


def _q8_1_values(xq):
    """The values of Q8_1 rows: every int8 times its block's f16 scale (exact in 32 bits)."""
    d = xq[..., 0:2].contiguous().view(torch.float16).float()
    q = xq[..., 4:36].contiguous().view(torch.int8).float()
    return (q * d).view(xq.shape[0], -1)


def _plain_norm(s):
    c = s["case"]
    x, res = s["x"].float(), None
    if s["res"] is not None:
        res = (x + s["res"].float()).to(s["res"].dtype)
        x = res.float()
    rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + c["eps"])
    n = x * rstd * (s["w"].float() + c["offset"])
    b = n.view(c["T"], -1, 32)
    d = b.abs().amax(-1, keepdim=True) / 127.0
    di = torch.where(d >= 2.0 ** -126, 1.0 / d, torch.zeros_like(d))
    q = torch.round(b * di).clamp(-128, 127)
    # the 8-bit rows as the values that they stand for, in the scale's own type
    values = (q * d.to(torch.float16).float()).view(c["T"], -1).to(torch.float16)
    return values, res, n.to(DTYPES[c["y"]]) if c["y"] else None


def _plain_route(s):
    c, T, E = s["case"], s["case"]["T"], s["case"]["E"]
    x = s["logits"].float()
    off = x.isnan() | (x == -math.inf)
    x = x.masked_fill(off, -math.inf)
    none = off.all(-1, keepdim=True)
    # the order of the experts in 64 bits, where near scores keep their order; without a bias it is that of the logits
    x64 = x.double()
    if c["scoring"] == "softmax":
        e = torch.exp(x64 - x64.amax(-1, keepdim=True).masked_fill(none, 0.0))
        score = e / e.sum(-1, keepdim=True).masked_fill(none, 1.0)
    else:
        score = 1.0 / (1.0 + torch.exp(-x64))
    pick = score + s["bias"].double() if s["bias"] is not None else score
    by = pick if s["bias"] is not None else x64
    if c["groups"] > 1:
        best = pick.masked_fill(off, -math.inf).view(T, c["groups"], -1).sort(dim=-1, descending=True).values[..., :2]
        if c["group_score"] == "max":
            best = (by.masked_fill(off, -math.inf)).view(T, c["groups"], -1).amax(-1)
        else:
            best = best[..., 0] + best[..., 1].masked_fill(best[..., 1] == -math.inf, 0.0)
        kept = best.sort(dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        inside = torch.zeros(T, c["groups"], dtype=torch.bool, device=x.device).scatter(1, kept, True)
        inside = inside.view(T, c["groups"], 1).expand(T, c["groups"], E // c["groups"]).reshape(T, E)
    else:
        inside = torch.ones_like(off)
    by = by.masked_fill(off, -1e300).masked_fill(~inside, -math.inf)
    ids = by.sort(dim=-1, descending=True, stable=True).indices[:, :c["top_k"]]
    chosen, lost = x.gather(1, ids), off.gather(1, ids)
    if c["scoring"] == "softmax":
        top = chosen.amax(-1, keepdim=True) if c["renorm"] else x.amax(-1, keepdim=True)
        top = top.masked_fill(top == -math.inf, 0.0)
        w = torch.exp(chosen - top)
        if not c["renorm"]:
            w = w / torch.exp(x - top).sum(-1, keepdim=True).masked_fill(none, 1.0)
    else:
        w = 1.0 / (1.0 + torch.exp(-chosen))
    w = w.masked_fill(lost, 0.0)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = w / total.masked_fill(total == 0.0, 1.0)
    return ids.to(torch.int32), w * c["scale"]


def _plain_matvec(s):
    c = s["case"]
    M, K, n = c["M"], c["K"], c["K"] // c["group"]
    q = torch.stack((s["w"] & 15, s["w"] >> 4), -1).view(M, n, c["group"]).float()
    if s["zeros"] is None:
        zero = 8.0
    else:
        zero = torch.stack((s["zeros"] & 15, s["zeros"] >> 4), -1).view(M, -1)[:, :n, None].float()
    W = ((q - zero) * s["scales"].float()[:, :, None]).view(M, K)
    return _q8_1_values(s["xq"]) @ W.t()


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "read":
        return _q8_1_values(state["xq"]).to(DTYPES[state["case"]["y"]])
    return _plain_route(state) if op == "route" else _plain_matvec(state)


# ---------------------------------------------------------------- in 64 bits


def _exact_q8_1(xq):
    """Q8_1 bytes read one field at a time, in 64 bits."""
    T, B = xq.shape[:2]
    bits = xq[..., 0].to(torch.int64) | (xq[..., 1].to(torch.int64) << 8)
    frac, power = (bits & 1023).double(), (bits >> 10) & 31
    d = torch.where(power == 0, frac * 2.0 ** -24, (1024.0 + frac) * torch.exp2(power.double() - 25.0))
    d = torch.where(bits >= 1 << 15, -d, d)
    q = xq[..., 4:36].to(torch.int64)
    q = torch.where(q > 127, q - 256, q)
    return torch.einsum("tbi,tb->tbi", q.double(), d).reshape(T, B * 32)


def _exact_norm(c, s):
    values, sums, rows = [], [], []
    for x, r in zip(s["x"].split(2048), s["res"].split(2048) if s["res"] is not None else [None] * c["T"]):
        h = x.double()
        if r is not None:
            h = (h + r.double()).to(r.dtype)
            sums.append(h)
            h = h.double()
        n = h * torch.rsqrt(h.pow(2).sum(1, keepdim=True) / c["K"] + c["eps"]) * (s["w"].double() + c["offset"])
        rows.append(n)
        b = n.reshape(-1, 32)
        top = b.abs().max(1).values
        step = (top / 127.0)[:, None]
        q = torch.where(step > 0, b / step, 0.0).round()
        values.append((q * step.half().double()).reshape(n.shape))
    return torch.cat(values), torch.cat(sums) if sums else None, torch.cat(rows) if c["y"] else None


def _exact_route(c, s):
    per = c["E"] // c["groups"]
    place = torch.arange(c["E"], device=s["logits"].device)
    all_ids, all_w = [], []

    def ranks(v):
        """How many come before each: those with more, and those before it with as much."""
        n = torch.arange(v.shape[1], device=v.device)
        more = v[:, None, :] > v[:, :, None]
        same = (v[:, None, :] == v[:, :, None]) & (n[None, None, :] < n[None, :, None])
        return (more | same).sum(-1)

    for x in s["logits"].double().split(2048):
        live = x > -math.inf
        z = torch.where(live, x, -1e4)
        if c["scoring"] == "softmax":
            e = torch.where(live, torch.exp(z - z.max(1, keepdim=True).values), 0.0)
            score = e / e.sum(1, keepdim=True).clamp_min(1e-300)
        else:
            score = torch.where(live, torch.sigmoid(z), 0.0)
        value = score if s["bias"] is None else score + s["bias"].double()
        order = torch.where(live, x if s["bias"] is None else value, -1e30)
        if c["groups"] > 1:
            grouped = lambda v: v.reshape(-1, c["groups"], per)  # noqa: E731
            if c["group_score"] == "max":
                g = grouped(order).max(-1).values
            else:
                r = ranks(grouped(torch.where(live, value, -1e30)).reshape(-1, per)).view(-1, c["groups"], per)
                two = (r < 2) & grouped(live)
                g = torch.where(two, grouped(value), 0.0).sum(-1)
                g = torch.where(grouped(live).any(-1), g, -1e30)
            kept = (ranks(g) < c["keep"]).repeat_interleave(per, 1)
            order = torch.where(kept, order, -1e60)
        rank = ranks(order)
        first = torch.where(rank < c["top_k"], rank, c["E"])
        ids = torch.zeros(x.shape[0], c["E"] + 1, dtype=torch.int64, device=x.device)
        ids = ids.scatter(1, first, place.expand_as(first))[:, :c["top_k"]]
        if c["renorm"] and c["scoring"] == "softmax":
            # of the chosen alone: the others' sum cancels
            zs = z.gather(1, ids)
            w = torch.where(live.gather(1, ids), torch.exp(zs - zs.max(1, keepdim=True).values), 0.0)
        else:
            w = score.gather(1, ids)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
        all_ids.append(ids)
        all_w.append(w * c["scale"])
    return torch.cat(all_ids).to(torch.int32), torch.cat(all_w)


def _exact_matvec(c, s):
    x = _exact_q8_1(s["xq"])
    rows = []
    at = torch.arange(c["K"], device=x.device)
    for i, w in zip(range(0, c["M"], 4096), s["w"].split(4096)):
        q = (w[:, at // 2].to(torch.int32) >> (4 * (at % 2)).to(torch.int32)) & 15
        if s["zeros"] is None:
            z = 8
        else:
            g = at // c["group"]
            z = (s["zeros"][i:i + 4096][:, g // 2].to(torch.int32) >> (4 * (g % 2)).to(torch.int32)) & 15
        scale = s["scales"][i:i + 4096].double()[:, at // c["group"]]
        rows.append(x @ ((q - z).double() * scale).t().contiguous())
    return torch.cat(rows, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "read":
        return _exact_q8_1(s["xq"])
    return _exact_route(case, s) if case["op"] == "route" else _exact_matvec(case, s)
