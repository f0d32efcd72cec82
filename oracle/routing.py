"""Routing of tokens to experts (oracle side).

TEST INFRASTRUCTURE ONLY (see the package docstring).

One token at a time, from the definition, in float64: scores, the bias that
only selects, groups of experts, the chosen in decreasing order with equal
values in the order of their index, and their weights.
"""
from __future__ import annotations

import numpy as np


def _best_first(values, index):
    """``index`` sorted by decreasing value, equal values by increasing index."""
    return sorted(index, key=lambda i: (-values[i], i))


def route(logits: np.ndarray, top_k: int, scoring: str = "softmax", bias=None, n_groups: int = 1,
          topk_groups: int = 1, group_score: str = "max", renormalize: bool = False, scale: float = 1.0):
    """``logits[T, E]`` -> (ids int32, weights float64), both ``[T, top_k]``.

    A logit that is -inf or NaN masks its expert; +inf counts as the largest
    float32.
    """
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    per = E // n_groups
    ids = np.zeros((T, top_k), np.int32)
    weights = np.zeros((T, top_k), np.float64)
    for t in range(T):
        row = np.minimum(x[t], float(np.finfo(np.float32).max))
        live = [e for e in range(E) if row[e] > -np.inf]
        alive = set(live)
        score = np.zeros(E)
        if live:
            if scoring == "softmax":
                p = np.exp(row[live] - row[live].max())
                score[live] = p / p.sum()
            else:
                with np.errstate(over="ignore"):
                    score[live] = 1.0 / (1.0 + np.exp(-row[live]))
        value = score + np.asarray(bias, np.float64) if bias is not None else score
        order = value if bias is not None else row
        groups = {}
        for g in range(n_groups):
            members = [e for e in live if e // per == g]
            if not members:
                groups[g] = -np.inf
            elif group_score == "max":
                groups[g] = max(order[e] for e in members)
            else:
                groups[g] = sum(sorted((value[e] for e in members), reverse=True)[:2])
        kept = set(_best_first(groups, range(n_groups))[:topk_groups])
        inside = [e for e in range(E) if e // per in kept]
        chosen = _best_first(order, [e for e in inside if e in alive])[:top_k]
        w = score[chosen]
        if renormalize and chosen:
            if scoring == "softmax":   # the other experts' sum cancels
                w = np.exp(row[chosen] - row[chosen].max())
            w = w / w.sum() if w.sum() > 0 else w
        weights[t, :len(chosen)] = w * scale
        chosen = chosen + [e for e in inside if e not in alive]
        ids[t] = chosen[:top_k]
    return ids, weights
