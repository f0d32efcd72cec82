"""Cases and plain forms of the attention half of a decoder layer.

Five operators are measured: the norm of queries and keys for each head with
the position rotation, appending keys and values to a paged cache of 4 bits a
value, reading that cache back, the attention of a few new tokens over it,
and the attention over whole prompts.  Each has a plain form here, made of
elementary torch operations in 32 bits, and an exact form in 64 bits.

Where ``own`` is true, ``run`` calls the library instead.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
HALF = ["f16", "bf16"]
HEAD = [64, 96, 128, 128, 128, 192, 256]

# The largest sizes that draw() gives: those of the largest listed case of each operator.
MOST_ROPE, MOST_APPEND, MOST_READ = 16384 * 72 * 128, 8192 * 8 * 128, 65536 * 8 * 128
MOST_CACHE, MOST_PROMPT = 64 * 8192 * 8 * 128, 2 * 32 * 128 * 6000 * 6000


def listed():
    return [
        # One decoded token: q and k of the fp32 product of the stacked projections.
        {"name": "rope 1x32+8x128", "op": "rope", "T": 1, "Hq": 32, "Hk": 8, "D": 128, "rot": 128, "x": "f32",
         "y": "bf16", "w": "bf16", "offset": 0.0, "pairs": "halves"},
        # A long prompt of a wide model.
        {"name": "rope 16384x64+8x128", "op": "rope", "T": 16384, "Hq": 64, "Hk": 8, "D": 128, "rot": 128, "x": "bf16",
         "y": "bf16", "w": "f32", "offset": 1.0, "pairs": "halves"},
        # The new tokens of a small decode batch, from the fp32 product, half of each head rotated.
        {"name": "append 5x8x128", "op": "append", "T": 5, "Hk": 8, "D": 128, "rot": 64, "x": "f32", "page": 16,
         "pairs": "neighbours"},
        # A prompt's keys and values.
        {"name": "append 8192x8x128", "op": "append", "T": 8192, "Hk": 8, "D": 128, "rot": 128, "x": "bf16",
         "page": 64, "pairs": "halves"},
        # The cached context of a prompt's next chunk: a short one of narrow heads, and a long one.
        {"name": "read 333x4x64", "op": "read", "T": 333, "Hk": 4, "D": 64, "page": 16, "y": "f16"},
        {"name": "read 65536x8x128", "op": "read", "T": 65536, "Hk": 8, "D": 128, "page": 64, "y": "bf16"},
        # One decoded token of one sequence.
        {"name": "cache 1x1000 32/8x128", "op": "cache", "B": 1, "n": 1, "Hq": 32, "Hk": 8, "D": 128, "len": 1000,
         "ragged": False, "page": 16, "window": 0, "x": "bf16"},
        # Four drafted tokens for each of a few sequences, ungrouped narrow heads, a sliding window.
        {"name": "cache 5x4x4099 16/16x64", "op": "cache", "B": 5, "n": 4, "Hq": 16, "Hk": 16, "D": 64, "len": 4099,
         "ragged": True, "page": 32, "window": 2000, "x": "f16"},
        # A full decode batch over contexts of different lengths.
        {"name": "cache 64x8192 32/8x128", "op": "cache", "B": 64, "n": 1, "Hq": 32, "Hk": 8, "D": 128, "len": 8192,
         "ragged": True, "page": 64, "window": 0, "x": "bf16"},
        # A few short prompts, one of them a single token.
        {"name": "prompt 1+17+130 8/2x64", "op": "prompt", "q": "1,17,130", "k": "1,17,130", "Hq": 8, "Hk": 2, "D": 64,
         "causal": True, "window": 0, "x": "f16"},
        # A chunk of a long prompt behind its context, wide heads.
        {"name": "prompt 512 of 4608 16/4x256", "op": "prompt", "q": "512", "k": "4608", "Hq": 16, "Hk": 4, "D": 256,
         "causal": True, "window": 0, "x": "bf16"},
        # Two long prompts packed.
        {"name": "prompt 6000+2192 32/8x128", "op": "prompt", "q": "6000,2192", "k": "6000,2192", "Hq": 32, "Hk": 8,
         "D": 128, "causal": True, "window": 0, "x": "bf16"},
    ]


def draw(rng):
    def spread(lo, hi):
        hi = max(lo, hi)
        return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    op = rng.choice(["rope", "append", "read", "cache", "cache", "prompt", "prompt"])
    D = rng.choice(HEAD)
    Hk = rng.choice([1, 2, 3, 4, 8, 8, 16])
    group = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16])
    rot = rng.choice([D, D, D, D // 2])
    pairs, page = rng.choice(["halves", "neighbours"]), rng.choice([16, 32, 64, 128])
    if op == "rope":
        w = rng.choice(["", "f32", "f16", "bf16"])
        return {"op": op, "T": spread(1, min(16384, MOST_ROPE // (Hk * (group + 1) * D))), "Hq": Hk * group, "Hk": Hk,
                "D": D, "rot": rot, "x": rng.choice(list(DTYPES)), "y": rng.choice(list(DTYPES)), "w": w,
                "offset": rng.choice([0.0, 1.0]) if w else 0.0, "pairs": pairs}
    if op == "append":
        return {"op": op, "T": spread(1, min(16384, MOST_APPEND // (Hk * D))), "Hk": Hk, "D": D,
                "rot": rng.choice([0, rot]), "x": rng.choice(list(DTYPES)), "page": page, "pairs": pairs}
    if op == "read":
        return {"op": op, "T": spread(1, min(65536, MOST_READ // (Hk * D))), "Hk": Hk, "D": D, "page": page,
                "y": rng.choice(list(DTYPES))}
    if op == "cache":
        B, n = spread(1, 64), rng.choice([1, 1, 1, 2, 3, 5, 8])
        length = spread(1, min(32768, MOST_CACHE // (B * Hk * D)))
        return {"op": op, "B": B, "n": n, "Hq": Hk * group, "Hk": Hk, "D": D, "len": length,
                "ragged": rng.choice([False, True]), "page": page,
                "window": rng.choice([0, 0, 0, max(1, length // 2)]), "x": rng.choice(HALF)}
    most = math.isqrt(MOST_PROMPT // (Hk * group * D))
    B = rng.choice([1, 1, 2, 3, 5])
    top = spread(1, min(8192, int(most / math.sqrt(B))))
    q = [top] + [rng.randint(1, top) for _ in range(B - 1)]
    rng.shuffle(q)
    causal = rng.choice([True, True, True, False])
    k, window = q, 0
    if causal and rng.choice([False, False, True]):
        k = [n + rng.randint(0, max(1, int(most / math.sqrt(B)) - n)) for n in q]
        if max(q) * max(k) * B * Hk * group * D > MOST_PROMPT:
            k = q
    if causal and rng.choice([False, False, True]):
        window = rng.randint(1, max(k))
    return {"op": op, "q": ",".join(map(str, q)), "k": ",".join(map(str, k)), "Hq": Hk * group, "Hk": Hk, "D": D,
            "causal": causal, "window": window, "x": rng.choice(HALF)}


def _lens(c):
    """The tokens in the cache for each sequence: those of the case, for a ragged batch from a quarter of it on."""
    if not c["ragged"]:
        return [c["len"]] * c["B"]
    r = random.Random(c["B"] * 100003 + c["len"])
    return [c["len"]] + [r.randint(c["len"] // 4, c["len"]) for _ in range(c["B"] - 1)]


def _pairs(q, k, causal, window):
    """How many (query, key) pairs of a sequence are visible."""
    if not causal:
        return q * k
    total = 0
    for i in range(q):
        n = max(0, k - q + i + 1)
        total += min(n, window) if window else n
    return total


def _ints(text):
    return [int(x) for x in text.split(",")]


def work(case):
    c, D = case, case["D"]
    if c["op"] == "rope":
        n = c["T"] * (c["Hq"] + c["Hk"]) * D
        return {"bytes": n * (SIZES[c["x"]] + SIZES[c["y"]]) + c["T"] * (4 * c["rot"] + 4)
                + (2 * D * SIZES[c["w"]] if c["w"] else 0), "flops": 7.0 * n}
    if c["op"] == "append":
        # the append, and reading the appended tokens back: 5 bits a value written and read, and a 16-bit value each
        n = 2 * c["T"] * c["Hk"] * D
        return {"bytes": n * (SIZES[c["x"]] + 2 * 0.625 + 2) + c["T"] * (4 * c["rot"] + 4 + 2 * 8), "flops": 10.0 * n}
    if c["op"] == "read":
        n = 2 * c["T"] * c["Hk"] * D
        return {"bytes": n * (0.625 + SIZES[c["y"]]) + 8 * c["T"], "flops": 2.0 * n}
    if c["op"] == "cache":
        seen = [min(n, c["window"] + c["n"] - 1) if c["window"] else n for n in _lens(c)]
        pairs = sum(_pairs(min(c["n"], n), n, True, c["window"]) for n in _lens(c))
        return {"bytes": sum(seen) * c["Hk"] * D * 2 * 0.625 + 2 * c["B"] * c["n"] * c["Hq"] * D * SIZES[c["x"]]
                + 4 * sum(-(-n // c["page"]) for n in seen), "flops": 4.0 * pairs * c["Hq"] * D}
    q, k = _ints(c["q"]), _ints(c["k"])
    pairs = sum(_pairs(a, b, c["causal"], c["window"]) for a, b in zip(q, k))
    return {"bytes": SIZES[c["x"]] * D * (2 * sum(q) * c["Hq"] + 2 * sum(k) * c["Hk"]), "flops": 4.0 * pairs * c["Hq"] * D}


# ---------------------------------------------------------------- inputs


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _below(g, high, *shape):
    return torch.randint(0, high, shape, generator=g, device=DEVICE)


def _table(positions, rot):
    """Rows of cosines and sines, from angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, device=DEVICE, dtype=torch.float64) / rot)
    a = torch.arange(positions, device=DEVICE, dtype=torch.float64)[:, None] * f
    return torch.cat((torch.cos(a), torch.sin(a)), 1).float()


def _heads(g, T, H, D):
    """Rows of heads with a few channels far larger than the rest, as keys have them."""
    loud = torch.where(_uniform(g, H, D) < 0.02, 6.0, 1.0)
    return _normal(g, T, H, D) * loud + 0.5 * _normal(g, H, D)


def _filled(g, pages, H, page, D):
    """A cache of random 4-bit values with scales that give them a spread of about one."""
    cells, nb = pages * H * (page // 16), D // 32
    c = _below(g, 256, cells, 20 * D).to(torch.uint8)

    def scales(*shape):
        d = 0.1 + 0.2 * _uniform(g, *shape)
        return d.half(), (-d * (7.5 + _normal(g, *shape))).half()

    d, m = scales(cells, nb * 16)
    c[:, 8 * D:10 * D] = torch.stack((d, m), -1).view(torch.uint8).view(cells, -1)
    d, m = scales(cells, 4, nb, 4)
    c[:, 18 * D:] = torch.cat((d, m), -1).view(torch.uint8).view(cells, -1)
    return c.view(pages, H, page // 16, 20 * D)


def prepare(case, seed):
    c, g = case, torch.Generator(device=DEVICE).manual_seed(seed)
    s, D = {"case": dict(c)}, c["D"]
    if c["op"] == "rope":
        # q and k as the stacked product leaves them, v behind them in each row
        x = _normal(g, c["T"], c["Hq"] + 2 * c["Hk"], D) * (0.5 + _uniform(g, c["Hq"] + 2 * c["Hk"], 1))
        x = x.to(DTYPES[c["x"]])
        s["q"], s["k"] = x[:, :c["Hq"]], x[:, c["Hq"]:c["Hq"] + c["Hk"]]
        s["wq"] = (1.0 - c["offset"] + 0.2 * _normal(g, D)).to(DTYPES[c["w"]]) if c["w"] else None
        s["wk"] = (1.0 - c["offset"] + 0.2 * _normal(g, D)).to(DTYPES[c["w"]]) if c["w"] else None
        first = int(_below(g, 4096, 1).item())
        s["rope"] = _table(4096 + c["T"], c["rot"])
        s["positions"] = first + torch.arange(c["T"], device=DEVICE, dtype=torch.int32)
    elif c["op"] == "append":
        x = torch.cat((_heads(g, c["T"], c["Hk"], D), _normal(g, c["T"], c["Hk"], D)), 1).to(DTYPES[c["x"]])
        s["k"], s["v"] = x[:, :c["Hk"]], x[:, c["Hk"]:]
        pages = -(-c["T"] // c["page"]) + 3
        s["cache"] = torch.zeros(pages, c["Hk"], c["page"] // 16, 20 * D, dtype=torch.uint8, device=DEVICE)
        # tokens in a row through shuffled pages, from inside a page on
        at = torch.randperm(pages, generator=g, device=DEVICE)
        t = torch.arange(c["T"], device=DEVICE) + int(_below(g, 2 * c["page"], 1).item())
        s["slots"] = at[t // c["page"]] * c["page"] + t % c["page"]
        s["rope"] = _table(4096 + c["T"], c["rot"]) if c["rot"] else None
        s["positions"] = (t + int(_below(g, 2048, 1).item())).clamp_max(4095 + c["T"]).to(torch.int32)
    elif c["op"] == "read":
        pages = -(-c["T"] // c["page"]) + 3
        s["cache"] = _filled(g, pages, c["Hk"], c["page"], D)
        at = torch.randperm(pages, generator=g, device=DEVICE)
        t = torch.arange(c["T"], device=DEVICE) + int(_below(g, 2 * c["page"], 1).item())
        s["slots"] = at[t // c["page"]] * c["page"] + t % c["page"]
    elif c["op"] == "cache":
        per = -(-c["len"] // c["page"])
        pages = c["B"] * per + 2
        s["cache"] = _filled(g, pages, c["Hk"], c["page"], D)
        s["table"] = torch.randperm(pages, generator=g, device=DEVICE)[:c["B"] * per].view(c["B"], per).to(torch.int32)
        s["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device=DEVICE)
        s["q"] = (1.2 * _normal(g, c["B"], c["n"], c["Hq"], D)).to(DTYPES[c["x"]])
    else:
        q, k = _ints(c["q"]), _ints(c["k"])
        t = DTYPES[c["x"]]
        s["q"] = (1.2 * _normal(g, sum(q), c["Hq"], D)).to(t)
        x = torch.cat((_heads(g, sum(k), c["Hk"], D) * 0.8, _normal(g, sum(k), c["Hk"], D)), 1).to(t)
        s["k"], s["v"] = x[:, :c["Hk"]], x[:, c["Hk"]:]
        s["cu_q"] = torch.tensor([0] + q, device=DEVICE).cumsum(0).to(torch.int32)
        s["cu_k"] = torch.tensor([0] + k, device=DEVICE).cumsum(0).to(torch.int32)
    return s


# ---------------------------------------------------------------- the library's calls


def _run_own(s):
    import quantized_matmul_q8_amd as qmm

    c = s["case"]
    if c["op"] == "rope":
        return qmm.qk_norm_rope(s["q"], s["k"], s["rope"], s["positions"], q_weight=s["wq"], k_weight=s["wk"], eps=1e-6,
                                weight_offset=c["offset"], interleaved=c["pairs"] == "neighbours", dtype=DTYPES[c["y"]])
    if c["op"] == "append":
        qmm.kv_append_q4(s["k"], s["v"], s["cache"], s["slots"], rope=s["rope"],
                         positions=s["positions"] if c["rot"] else None, interleaved=c["pairs"] == "neighbours")
        return qmm.kv_read_q4(s["cache"], s["slots"], torch.float16)
    if c["op"] == "read":
        return qmm.kv_read_q4(s["cache"], s["slots"], DTYPES[c["y"]])
    if c["op"] == "cache":
        return qmm.attn_q4(s["q"], s["cache"], s["table"], s["lens"], window=c["window"])
    return qmm.attn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=c["causal"], window=c["window"])


# ---------------------------------------------------------------- plain forms


def _rotated(x, rope, positions, pairs):
    """x [T, H, D] with its first dims turned by the table's angles, every product and sum rounded to 32 bits."""
    rot = rope.shape[1]
    cos, sin = rope[positions.long()].view(-1, 1, 2, rot // 2).unbind(2)
    r = x[..., :rot]
    a, b = (r[..., :rot // 2], r[..., rot // 2:]) if pairs == "halves" else (r[..., 0::2], r[..., 1::2])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.cat((u, v), -1) if pairs == "halves" else torch.stack((u, v), -1).flatten(-2)
    return torch.cat((r, x[..., rot:]), -1)


def _plain_rope(s):
    c = s["case"]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)) * (w.float() + c["offset"])
        return _rotated(x, s["rope"], s["positions"], c["pairs"]).to(DTYPES[c["y"]])

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _four_bits(x):
    """Blocks of 32 as 4-bit steps above their least value, with 16-bit scales: the values that they stand for."""
    b = x.nan_to_num(0.0, 32768.0, -32768.0).clamp(-32768.0, 32768.0).unflatten(-1, (-1, 32))
    lo, hi = b.amin(-1, keepdim=True), b.amax(-1, keepdim=True)
    d = ((hi - lo) / torch.full_like(lo, 15.0)).half().float()
    m = lo.half().float()
    inv = torch.where(d > 0, torch.ones_like(d) / d, torch.zeros_like(d))
    n = torch.round((b - m) * inv).clamp(0.0, 15.0)
    return (n * d + m).half().flatten(-2)


def _plain_append(s):
    k = s["k"].float()
    if s["rope"] is not None:
        k = _rotated(k, s["rope"], s["positions"], s["case"]["pairs"])
    return _four_bits(k), _four_bits(s["v"].float())


def _plain_cells(cells, D):
    """Cells [..., 20 D] of 16 tokens -> their keys and values [..., 16, D] in 32 bits."""
    nb, lead = D // 32, cells.shape[:-1]
    kn, ks, vn, vs = cells.split((8 * D, 2 * D, 8 * D, 2 * D), -1)
    # keys: byte 4j of a block holds values 8j and 8j + 2, the next 8j + 4 and 8j + 6, then the odd ones
    kn = kn.reshape(*lead, nb, 16, 4, 2, 2)
    kn = torch.stack((kn & 15, kn >> 4), -1)                       # [nb, token, j, odd, half, step]
    kn = kn.movedim(-3, -1).reshape(*lead, nb, 16, 32).float()
    ks = ks.contiguous().view(torch.float16).reshape(*lead, nb, 16, 2).float()
    k = (kn * ks[..., 0:1] + ks[..., 1:2]).half().float()
    k = k.transpose(-3, -2).reshape(*lead, 16, D)
    # values: of a quad of tokens the bytes hold tokens 0, 2, 1, 3, and dims c and c + 16 of the block
    vn = vn.reshape(*lead, 4, 16, nb, 2, 2)
    vn = torch.stack((vn & 15, vn >> 4), -1)                       # [quad, c, nb, odd, pair, upper]
    vn = vn.permute(*range(len(lead)), *(len(lead) + i for i in (0, 4, 3, 2, 5, 1))).reshape(*lead, 4, 4, nb, 32).float()
    vs = vs.contiguous().view(torch.float16).reshape(*lead, 4, nb, 2, 4).float()
    vs = vs.movedim(-1, -3)[..., None]                             # [quad, token, nb, (d, m), 1]
    v = (vn * vs[..., 0, :] + vs[..., 1, :]).half().float()
    return k, v.reshape(*lead, 16, D)


def _plain_read(s):
    c = s["case"]
    k, v = _plain_cells(s["cache"], c["D"])                        # [pages, H, cells, 16, D]
    pick = lambda x: x.permute(0, 2, 3, 1, 4).reshape(-1, c["Hk"], c["D"])[s["slots"]].to(DTYPES[c["y"]])  # noqa: E731
    return pick(k), pick(v)


def _softmax(x):
    """Over the last dim; rows of -inf give zeros."""
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top.masked_fill(top == -math.inf, 0.0))
    return e / e.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain_cache(s):
    c = s["case"]
    B, n, Hk, D, g = c["B"], c["n"], c["Hk"], c["D"], c["Hq"] // c["Hk"]
    cells = s["cache"][s["table"].long()]                          # [B, pages, H, cells, bytes]
    k, v = _plain_cells(cells.transpose(1, 2), D)
    k, v = k.reshape(B, Hk, -1, D), v.reshape(B, Hk, -1, D)
    q = s["q"].float().view(B, n, Hk, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, n * g, D)
    x = torch.matmul(q, k.transpose(-1, -2).contiguous()).view(B, Hk, n, g, -1) / math.sqrt(D)
    at = s["lens"].view(B, 1, 1, 1, 1) - n + torch.arange(n, device=q.device).view(1, 1, n, 1, 1)
    j = torch.arange(k.shape[2], device=q.device)
    seen = j <= at
    if c["window"]:
        seen = seen & (j > at - c["window"])
    p = _softmax(x.masked_fill(~seen, -math.inf)).view(B, Hk, n * g, -1)
    y = torch.matmul(p, v).view(B, Hk, n, g, D).permute(0, 2, 1, 3, 4)
    return y.reshape(B, n, c["Hq"], D).to(s["q"].dtype)


def _plain_prompt(s):
    c = s["case"]
    Hk, D, g = c["Hk"], c["D"], c["Hq"] // c["Hk"]
    B, Lq, Lk = len(_ints(c["q"])), max(_ints(c["q"])), max(_ints(c["k"]))
    nq, nk = s["cu_q"].diff().view(B, 1), s["cu_k"].diff().view(B, 1)
    i, j = torch.arange(Lq, device=DEVICE), torch.arange(Lk, device=DEVICE)
    # the packed rows as padded sequences
    rows = (s["cu_q"][:-1, None] + i).clamp_max(s["q"].shape[0] - 1)
    cols = (s["cu_k"][:-1, None] + j).clamp_max(s["k"].shape[0] - 1)
    q = s["q"][rows].float().view(B, Lq, Hk, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, g * Lq, D)
    k = s["k"][cols].float().permute(0, 2, 3, 1).contiguous()
    v = s["v"][cols].float().transpose(1, 2).contiguous()
    x = torch.matmul(q, k).view(B, Hk, g, Lq, Lk) / math.sqrt(D)
    seen = (j < nk)[:, None]
    if c["causal"]:
        at = (nk - nq + i)[:, :, None]
        seen = seen & (j <= at)
        if c["window"]:
            seen = seen & (j > at - c["window"])
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    y = torch.matmul(_softmax(x).view(B, Hk, g * Lq, Lk), v).view(B, Hk, g, Lq, D).permute(0, 3, 1, 2, 4)
    return y.reshape(B, Lq, c["Hq"], D)[i < nq].to(s["q"].dtype)


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "append": _plain_append, "read": _plain_read, "cache": _plain_cache,
            "prompt": _plain_prompt}[state["case"]["op"]](state)


# ---------------------------------------------------------------- in 64 bits


def _exact_turn(x, rope, positions, pairs):
    rot = rope.shape[1]
    w = torch.complex(*(t.double() for t in rope[positions.long()].split(rot // 2, 1)))[:, None]
    y = x.clone()
    if pairs == "halves":
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot].contiguous()) * w
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * w
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def _exact_rope(c, s):
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        rows = []
        for at, part in zip(range(0, c["T"], 2048), x.split(2048)):
            h = part.double()
            if w is not None:
                h = h * torch.rsqrt(h.pow(2).sum(-1, keepdim=True) / c["D"] + 1e-6) * (w.double() + c["offset"])
            rows.append(_exact_turn(h, s["rope"], s["positions"][at:at + 2048], c["pairs"]))
        out.append(torch.cat(rows))
    return tuple(out)


def _exact_append(c, s):
    out = []
    for x, turn in ((s["k"].double(), c["rot"] > 0), (s["v"].double(), False)):
        if turn:
            x = _exact_turn(x, s["rope"], s["positions"], c["pairs"])
        b = x.reshape(-1, 32).clamp(-32768, 32768)
        lo = b.min(1).values
        step = ((b.max(1).values - lo) / 15).half().double()
        low = lo.half().double()
        n = torch.where(step[:, None] > 0, (b - low[:, None]) / step[:, None], 0.0).round().clamp(0, 15)
        out.append((low[:, None] + n * step[:, None]).half().double().view_as(x))
    return tuple(out)


def _exact_tokens(cache, D, slots):
    """The keys and values [H, slots, D] of cached tokens, each value looked up by its place in the bytes."""
    pages, H, cells = cache.shape[:3]
    flat, nb = cache.reshape(-1), D // 32
    cell, t = slots // 16, slots % 16
    base = ((cell // cells * H)[None] + torch.arange(H, device=slots.device)[:, None]) * cells + (cell % cells)[None]
    base = (base * 20 * D)[..., None]
    d = torch.arange(D, device=slots.device)
    b, r, t = d // 32, d % 32, t[None, :, None]

    def half(at):
        bits = flat[at].to(torch.int64) | flat[at + 1].to(torch.int64) << 8
        e, f, sign = bits >> 10 & 31, (bits & 1023).double(), torch.where(bits >= 32768, -1.0, 1.0).double()
        return sign * torch.where(e == 0, f * 2.0 ** -24, (1024 + f) * torch.exp2(e.double() - 25))

    low = lambda at: flat[at].to(torch.int64) & 15  # noqa: E731
    high = lambda at: flat[at].to(torch.int64) >> 4  # noqa: E731
    e = r % 8
    at = base + (b * 16 + t) * 16 + r // 8 * 4 + e % 2 * 2 + e // 4
    n = torch.where(e % 4 >= 2, high(at), low(at)).double()
    at = base + 8 * D + (b * 16 + t) * 4
    k = (n * half(at) + half(at + 2)).half().double()
    order = torch.tensor([0, 2, 1, 3], device=slots.device)[t % 4]
    at = base + 10 * D + ((t // 4 * 16 + r % 16) * nb + b) * 4 + order
    n = torch.where(r >= 16, high(at), low(at)).double()
    at = base + 18 * D + (t // 4 * nb + b) * 16 + t % 4 * 2
    return k, (n * half(at) + half(at + 8)).half().double()


def _exact_read(c, s):
    parts = [_exact_tokens(s["cache"], c["D"], x) for x in s["slots"].split(4096)]
    return tuple(torch.cat([p[i] for p in parts], 1).transpose(0, 1) for i in (0, 1))


def _exact_attention(q, k, v, causal, window):
    """q [n, D], k, v [L, D] -> [n, D]; the last query stands at the last key."""
    n, L = q.shape[0], k.shape[0]
    x = (q @ k.t().contiguous()) * q.shape[1] ** -0.5
    if causal:
        at = torch.arange(n, device=q.device)[:, None] + (L - n)
        j = torch.arange(L, device=q.device)[None]
        hidden = j > at
        if window:
            hidden = hidden | (j <= at - window)
        x = x.masked_fill(hidden, -math.inf)
    return torch.softmax(x, -1).nan_to_num(0.0) @ v


def _exact_cache(c, s):
    B, n, g = c["B"], c["n"], c["Hq"] // c["Hk"]
    y = torch.zeros(B, n, c["Hq"], c["D"], dtype=torch.float64, device=DEVICE)
    for b, L in enumerate(_lens(c)):
        t = torch.arange(L, device=DEVICE)
        slots = s["table"][b].long()[t // c["page"]] * c["page"] + t % c["page"]
        k, v = _exact_tokens(s["cache"], c["D"], slots)
        for h in range(c["Hq"]):
            y[b, :, h] = _exact_attention(s["q"][b, :, h].double(), k[h // g], v[h // g], True, c["window"])
    return y


def _exact_prompt(c, s):
    g = c["Hq"] // c["Hk"]
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    a = b = 0
    for n, L in zip(_ints(c["q"]), _ints(c["k"])):
        for h in range(c["Hq"]):
            y[a:a + n, h] = _exact_attention(s["q"][a:a + n, h].double(), s["k"][b:b + L, h // g].double(),
                                             s["v"][b:b + L, h // g].double(), c["causal"], c["window"])
        a, b = a + n, b + L
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "read": _exact_read, "cache": _exact_cache,
            "prompt": _exact_prompt}[case["op"]](case, s)
