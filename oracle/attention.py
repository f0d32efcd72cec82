"""Norm and rotation of heads, the 4-bit key-value cache, and attention (oracle side).

TEST INFRASTRUCTURE ONLY (see the package docstring).

Float64 throughout, but for the cache's bytes: their quantizer is emulated step
by step in IEEE float32, since they are compared bit for bit.  The cache is
addressed one code at a time, by the places that the layout gives each.
"""
from __future__ import annotations

import numpy as np

F32 = np.float32


def rope_table(positions: int, rot: int, base: float = 10000.0) -> np.ndarray:
    """fp32 [positions, rot]: cosines, then sines."""
    a = np.arange(positions)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate((np.cos(a), np.sin(a)), 1).astype(F32)


def turn(x: np.ndarray, table: np.ndarray, positions: np.ndarray, interleaved: bool) -> np.ndarray:
    """Heads ``x[T, H, D]`` with their pairs turned, every product and sum in x's own precision."""
    rot = table.shape[1]
    rows = table[np.clip(positions, 0, table.shape[0] - 1)].astype(x.dtype)[:, None, :]
    c, s = rows[..., :rot // 2], rows[..., rot // 2:]
    ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(rot // 2), np.arange(rot // 2, rot))
    a, b, y = x[..., ia], x[..., ib], x.copy()
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def head_norm(x: np.ndarray, w: np.ndarray, eps: float, offset: float = 0.0) -> np.ndarray:
    x = np.asarray(x, np.float64)
    ms = (x * x).sum(-1, keepdims=True) / x.shape[-1]
    rms = np.where(ms + eps == 0, 1.0, np.sqrt(ms + eps))       # a head of zeros stays zeros
    return x / rms * (np.asarray(w, np.float64) + offset)


def q4_blocks(x: np.ndarray):
    """fp32 ``x[..., D]`` -> codes [..., D], d and m [..., D/32] as f16: the steps of kv_append_q4."""
    x = np.asarray(x, F32)
    b = np.clip(np.where(np.isnan(x), F32(0), x), F32(-32768), F32(32768)).reshape(*x.shape[:-1], -1, 32)
    lo, hi = b.min(-1) + F32(0), b.max(-1) + F32(0)              # no minus zero
    d, m = ((hi - lo) / F32(15)).astype(np.float16), lo.astype(np.float16)
    df = d.astype(F32)
    with np.errstate(divide="ignore"):
        inv = np.where(df > 0, F32(1) / df, F32(0)).astype(F32)
    n = np.clip(np.rint((b - m.astype(F32)[..., None]) * inv[..., None]), 0, 15).astype(np.uint8)
    return n.reshape(x.shape), d, m


def q4_values(n: np.ndarray, d: np.ndarray, m: np.ndarray) -> np.ndarray:
    """The f16 numbers that codes stand for (n * d + m is exact in float64)."""
    r = lambda v: np.repeat(v.astype(np.float64), 32, -1)  # noqa: E731
    return (n * r(d) + r(m)).astype(np.float16)


def _places(D: int, t: int):
    """For token t of a cell, per value: byte and shift of the key's code and the value's; per block: byte of the
    key's (d, m), and of the value's d (its m is 8 bytes further)."""
    v = np.arange(D)
    b, e, nb = v // 32, v % 8, D // 32
    kb = (b * 16 + t) * 16 + v % 32 // 8 * 4 + (e % 2) * 2 + e // 4
    kshift = np.where(e % 4 >= 2, 4, 0)
    order = (0, 2, 1, 3)[t % 4]
    vb = 10 * D + ((t // 4 * 16 + v % 16) * nb + b) * 4 + order
    vshift = np.where(v % 32 >= 16, 4, 0)
    blk = np.arange(nb)
    return kb, kshift, vb, vshift, 8 * D + (blk * 16 + t) * 4, 18 * D + (t // 4 * nb + blk) * 16 + t % 4 * 2


def cache_store(cache: np.ndarray, slots, k: np.ndarray, v: np.ndarray) -> None:
    """Appends fp32 ``k[T, Hk, D]`` (turned already) and ``v`` into ``cache[pages, Hk, page/16, 20 D]``."""
    pages, Hk, cells, size = cache.shape
    D = size // 20
    parts = q4_blocks(k), q4_blocks(v)
    for i, slot in enumerate(np.asarray(slots)):
        if slot < 0 or slot >= pages * cells * 16:
            continue
        pg, at = divmod(int(slot), cells * 16)
        kb, ksh, vb, vsh, kd, vd = _places(D, at % 16)
        for h in range(Hk):
            cell = cache[pg, h, at // 16]
            for (n, d, m), byte, sh in ((parts[0], kb, ksh), (parts[1], vb, vsh)):
                for s in (0, 4):
                    w = sh == s
                    cell[byte[w]] = (cell[byte[w]] & (0xF0 if s == 0 else 0x0F)) | (n[i, h][w] << s)
            for (n, d, m), at0, at1 in ((parts[0], kd, kd + 2), (parts[1], vd, vd + 8)):
                for x, a in ((d[i, h], at0), (m[i, h], at1)):
                    raw = np.ascontiguousarray(x).view(np.uint8).reshape(-1, 2)
                    cell[a], cell[a + 1] = raw[:, 0], raw[:, 1]


def cache_load(cache: np.ndarray, slots):
    """The f16 keys and values [T, Hk, D] of the slots; zeros for slots outside the cache."""
    pages, Hk, cells, size = cache.shape
    D = size // 20
    k = np.zeros((len(slots), Hk, D), np.float16)
    v = k.copy()
    half = lambda cell, a: (cell[:, a].astype(np.uint16) | cell[:, a + 1].astype(np.uint16) << 8).view(np.float16)  # noqa: E731
    for i, slot in enumerate(np.asarray(slots)):
        if slot < 0 or slot >= pages * cells * 16:
            continue
        pg, at = divmod(int(slot), cells * 16)
        kb, ksh, vb, vsh, kd, vd = _places(D, at % 16)
        cell = cache[pg, :, at // 16]
        k[i] = q4_values((cell[:, kb] >> ksh) & 15, half(cell, kd), half(cell, kd + 2))
        v[i] = q4_values((cell[:, vb] >> vsh) & 15, half(cell, vd), half(cell, vd + 8))
    return k, v


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, seen: np.ndarray):
    """``q[n, Hq, D]``, ``k``, ``v`` [L, Hk, D], ``seen[n, L]`` -> (y, spread): the float64 result, and sum p |v| per
    element.  Queries that see nothing (or nothing above -inf) give zeros; keys that are not seen have no influence."""
    n, Hq, D = q.shape
    g = Hq // k.shape[1]
    y, spread = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    for h in range(Hq):
        kk, vv = k[:, h // g].astype(np.float64), v[:, h // g].astype(np.float64)
        for i in range(n):
            s = seen[i]
            if not s.any():
                continue
            with np.errstate(invalid="ignore"):
                x = kk[s] @ q[i, h].astype(np.float64) * scale
                if np.all(x == -np.inf):
                    continue
                p = np.exp(x - x.max())
                p /= p.sum()
                y[i, h], spread[i, h] = p @ vv[s], p @ np.abs(vv[s])
    return y, spread


def visible(n: int, L: int, causal: bool, window: int = 0) -> np.ndarray:
    """bool [n, L]: which keys each query sees; the last query stands at the last key."""
    at, j = np.arange(n)[:, None] + (L - n), np.arange(L)[None]
    seen = np.ones((n, L), bool)
    if causal:
        seen = j <= at
        if window:
            seen &= j > at - window
    return seen
