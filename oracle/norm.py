"""Root-mean-square norm with a residual (oracle side).

TEST INFRASTRUCTURE ONLY (see the package docstring).

``n = h / sqrt(mean(h^2) + eps) * (weight + offset)`` in float64, where ``h``
is the row as the residual stream stores it.  The Q8_1 rows of a fp32 ``n``
are those of ``quantize_q8_1``.
"""
from __future__ import annotations

import numpy as np


def rms_norm(h: np.ndarray, weight: np.ndarray, eps: float, offset: float = 0.0) -> np.ndarray:
    """Rows of ``h[T, K]`` (float64), each over its root mean square, times ``weight + offset``."""
    h = np.asarray(h, np.float64)
    ms = (h * h).sum(axis=1, keepdims=True) / h.shape[1]
    with np.errstate(divide="ignore", invalid="ignore"):
        return h / np.sqrt(ms + eps) * (np.asarray(weight, np.float64) + offset)
