"""The router's choice in fp64, one token and one expert at a time (the
definition in include/moe_w4a4.h, moe_w4a4_router)."""
from __future__ import annotations

import math

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)


def scores(row, scoring: str) -> list:
    """fp64 score of each logit of one token; None where it is masked."""
    seen = [None if math.isnan(v) or v == -math.inf else min(float(v), FLT_MAX) for v in row]
    live = [v for v in seen if v is not None]
    if scoring == "softmax":
        top = max(live, default=0.0)
        total = math.fsum(math.exp(v - top) for v in live)
        return [None if v is None else math.exp(v - top) / total for v in seen]
    if scoring == "sigmoid":
        return [None if v is None else (1 / (1 + math.exp(-v)) if v > -700 else 0.0) for v in seen]
    return [None if v is None else math.sqrt(max(v, 0.0) + math.log1p(math.exp(-abs(v)))) for v in seen]


def route_logits(logits, topk: int, scoring: str, bias=None, num_groups: int = 1, topk_groups: int = 1,
                 renormalize: bool = True, scale: float = 1.0):
    """(ids int32 [T, k], weights fp64 [T, k])."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    size = E // num_groups
    ids = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    for t in range(T):
        s = scores(logits[t], scoring)
        c = {}
        for e in range(E):
            if s[e] is None:
                continue
            v = (min(float(np.float32(logits[t, e])), FLT_MAX) if bias is None
                 else float(np.float32(np.float32(s[e]) + np.float32(bias[e]))))
            if v > -math.inf:                              # false for NaN
                c[e] = v
        if num_groups > 1:
            rank = []
            for g in range(num_groups):
                best = sorted((c[e] for e in range(g * size, (g + 1) * size) if e in c), reverse=True)
                if not best:
                    rank.append(-math.inf)
                elif bias is None or len(best) == 1:
                    rank.append(best[0])
                else:
                    rank.append(float(np.float32(best[0]) + np.float32(best[1])))
            kept = sorted(range(num_groups), key=lambda g: (-rank[g], g))[:topk_groups]
            c = {e: v for e, v in c.items() if e // size in kept}
        chosen = sorted(c, key=lambda e: (-c[e], e))[:topk]
        ids[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = [s[e] for e in chosen]
    if renormalize:
        w = w / (w.sum(axis=1, keepdims=True) + 1e-20)
    return ids, w * float(np.float32(scale))
