"""The allowed error of an attention kernel's output, shared by the attention tests.

A score is a sum of D products of 16-bit numbers, exact in fp32, in any order:
at most D + 8 roundings of 2^-24 of sum |q||k| scale, with those of the scale's
product and of the exponent's argument.  The exponential itself is right to
2^-21 relative (two units of its last place and its argument's).  So a term of
the softmax is off by its score's error and that, the term meets the values
rounded to 16 bits (half a step: 2^-11 relative in f16, with 10 bits of fraction,
2^-8 in bf16, with 7; or below 2^-30 of the largest), and the sums over n keys add at most n + 64 roundings.  Terms and
their sum are off alike, so twice; the error of y is that times sum p |v|.
"""
import numpy as np
import torch

U = 2.0**-24
HALF_STEP = {torch.float32: 2.0**-24, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
LEAST = {torch.float32: 2.0**-126, torch.float16: 2.0**-25, torch.bfloat16: 2.0**-126}


def allowed(q, k, scale, seen, y, spread, term, yt):
    """q [n, Hq, D], k [L, Hk, D] (numpy), seen [n, L]; `term`: the relative rounding of a term."""
    n, Hq, D = q.shape
    g = Hq // k.shape[1]
    size = np.zeros((n, Hq))
    for h in range(Hq):
        kk = np.where(np.isfinite(k[:, h // g]), np.abs(k[:, h // g].astype(np.float64)), 0.0)
        s = np.where(seen, np.abs(q[:, h].astype(np.float64)) @ kk.T, 0.0)
        size[:, h] = s.max(1, initial=0.0) * abs(scale)
    keys = seen.sum(1)[:, None]
    rel = 2 * ((D + 8) * U * size + 2.0**-21) + term + 2.0**-30 * keys + 2 * (keys + 64) * U
    err = rel[..., None] * spread
    return err + HALF_STEP[yt] * (np.abs(y) + err) + LEAST[yt]
