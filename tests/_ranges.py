"""Inputs and tolerances for attention where finite inputs stand at the ends of their ranges, shared by the tests.

Scores of 2^20 and more leave fp32 few bits or none behind the point, so random
inputs could be held to nothing.  Here every product q . k is a whole number of
quarters below 2^22 (of halves below 2^23 where D > 128) times a power of two,
which fp32 sums without rounding in any order: scores that differ at all differ
by what the inputs say.  A term is then off by the roundings of its own
difference to the largest score alone (of the scale times log2 e, twice, of the
product and of the exponent's argument: 4 * 2^-24 of the difference) and by the
exponential (2^-21: _attention.py), and so is each factor by which sums are
brought to a new maximum or joined, one for every level of score at the most and
two for waves and splits.  A difference of more than 60 leaves less than the
2^-30 that a small term may lose anyway.
"""
import numpy as np

import oracle
from _attention import HALF_STEP, LEAST, U
from _gpu import dev


def ints(x):
    return dev(np.array(x, np.int32))


def compare(y, q, k, v, scale, seen, count, term, yt):
    """y against the oracle; `count`: how many different scores a query meets."""
    ref, spread = oracle.attention(q, k, v, scale, seen)
    keys = seen.sum(1)[:, None, None]
    rel = 2 * (count + 3) * (4 * 60 * U + 2.0**-21) + term + 2.0**-30 * keys + 2 * (keys + 64) * U
    tol = rel * spread
    tol += HALF_STEP[yt] * (np.abs(ref) + tol) + LEAST[yt]
    got = y.double().cpu().numpy()
    assert np.all(np.isfinite(got)), np.argwhere(~np.isfinite(got))[:4].tolist()
    bad = np.abs(got - ref) - tol
    assert np.all(bad <= 0), (float(bad.max()), np.argwhere(bad > 0)[:4].tolist())


def levels(g, D, *shape):
    """Six levels, a quarter or a half apart."""
    return g.integers(0, 6, shape) / (4 if D <= 128 else 2)
