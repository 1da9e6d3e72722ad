"""Routing with a gate, oracle side (test infrastructure only): one token at a time, in Python floats.

The definition is the C ABI's (include/qtip_moe.h, "routing with a gate"); every choice is a sort by
(-value, index).
"""
from __future__ import annotations

import math

import numpy as np


def scores(row, score: str):
    """Scores of one token's logits; NaN logits score NaN, which is never chosen."""
    if score == "sigmoid":
        return [1.0 / (1.0 + math.exp(-v)) if v >= 0 else math.exp(v) / (1.0 + math.exp(v)) for v in row]
    num = [v for v in row if not math.isnan(v)]
    top = max(num, default=-math.inf)
    if top == -math.inf:
        return [math.nan if math.isnan(v) else 0.0 for v in row]
    ex = [math.nan if math.isnan(v) else 1.0 if v == top else math.exp(v - top) if math.isfinite(top) else 0.0
          for v in row]
    z = math.fsum(v for v in ex if not math.isnan(v))
    return [v / z for v in ex]


def shares(chosen, w, top):
    """The chosen scores w divided by their sum, from their logits where fp64 does not hold the scores:
    both kinds then go like exp(logit).  top: a softmax's largest logit, a sigmoid's 0."""
    z = math.fsum(w)
    if z > 1e-250:
        return [v / z for v in w]
    largest = max(chosen, default=-math.inf)
    if not largest - top >= -745.0:                # scores below exp(-745) count as 0
        return [0.0] * len(w)
    ex = [math.exp(v - largest) for v in chosen]
    return [v / math.fsum(ex) for v in ex]


def route_token(row, bias, k, score="softmax", num_groups=1, top_groups=1, group_top=1, renormalise=1, scale=1.0):
    row = [float(v) for v in row]
    E = len(row)
    s = scores(row, score)
    c = [s[e] + float(bias[e]) if bias is not None else s[e] for e in range(E)]
    able = [row[e] > -math.inf and c[e] > -math.inf for e in range(E)]   # NaN compares false
    size = E // num_groups
    if num_groups > 1:
        value = []
        for g in range(num_groups):
            best = sorted((c[e] for e in range(g * size, (g + 1) * size) if able[e]), reverse=True)[:group_top]
            value.append(sum(best) if best else -math.inf)
        kept = sorted((g for g in range(num_groups) if value[g] > -math.inf),
                      key=lambda g: (-value[g], g))[:top_groups]
        able = [able[e] and e // size in kept for e in range(E)]
    idx = sorted((e for e in range(E) if able[e]), key=lambda e: (-c[e], e))[:k]
    w = [s[e] for e in idx]
    if renormalise:
        top = 0.0 if score == "sigmoid" else max((v for v in row if not math.isnan(v)), default=0.0)
        w = shares([row[e] for e in idx], w, top)
    gap = k - len(idx)
    return idx + [-1] * gap, [v * scale for v in w] + [0.0] * gap


def route(logits, bias, k, **gate):
    out = [route_token(r, bias, k, **gate) for r in np.asarray(logits, np.float64)]
    return np.array([o[0] for o in out], np.int32), np.array([o[1] for o in out], np.float64)


def bins(topk_idx, num_experts):
    """(counts, offsets, pair ids in expert order, ascending within an expert); id -1 is in no bin."""
    flat = np.asarray(topk_idx).reshape(-1)
    members = [np.flatnonzero(flat == e) for e in range(num_experts)]
    counts = np.array([len(m) for m in members], np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return counts, offsets, np.concatenate(members).astype(np.int32)
