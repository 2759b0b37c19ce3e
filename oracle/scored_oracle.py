"""CPU oracle (fp64) of routing by scores: scores, groups, choice and weights
of one token after the other, by sorting.

Pinned by tests/test_scored_cpu.py: hand-worked groups and ties, the plain
top-k softmax router as a special case, a brute force over all subsets.
"""
from __future__ import annotations

import numpy as np


def scores(l, score):
    """fp64 scores [E] of one token's logits."""
    l = np.asarray(l, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        if np.all(l == -np.inf):
            return np.zeros_like(l)
        m = np.nan if np.isnan(l).any() else l.max()
        e = np.exp(l - m)
        return e / e.sum()


def route_scored(logits, k, score="sigmoid", bias=None, n_group=1, topk_group=None, group_best=2,
                 renormalize=True, scale=1.0):
    """(ids int32 [T][k], w fp64 [T][k])."""
    logits = np.asarray(logits)
    T, E = logits.shape
    size = E // n_group
    topk_group = n_group if topk_group is None else topk_group
    ids, w = np.zeros((T, k), dtype=np.int32), np.zeros((T, k))
    for t in range(T):
        s = scores(logits[t], score)
        c = s if bias is None else s + np.asarray(bias, dtype=np.float64)
        c = np.where(np.isnan(c), -np.inf, c)
        value = [sum(sorted(c[g * size:(g + 1) * size], reverse=True)[:group_best])
                 for g in range(n_group)]
        groups = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
        among = [e for g in groups for e in range(g * size, (g + 1) * size)]
        ids[t] = sorted(among, key=lambda e: (-c[e], e))[:k]
        w[t] = s[ids[t]]
        if renormalize:
            total = 0.0
            for v in w[t]:
                total += v
            w[t] = 0.0 if total == 0 else w[t] / total
        w[t] *= float(np.float32(scale))
    return ids, w
