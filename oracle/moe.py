"""Routing of tokens to experts, its gradient, and the choices grouped by expert: one token, one expert at a time.

Test infrastructure only (see the package docstring).
"""
from __future__ import annotations

import math

import numpy as np


def scores(logits, score: str):
    """The 64-bit scores of one token's logits (masked ones, -inf: 0)."""
    l = [float(v) for v in logits]
    if score == "sigmoid":
        return [0.0 if v == -math.inf else 1.0 if v == math.inf else 1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v in l]
    high = max(l)
    if high == -math.inf:
        return [0.0] * len(l)
    e = [math.exp(v - high) for v in l]
    total = math.fsum(e)
    return [v / total for v in e]


def route_token(logits, top, score="softmax", bias=None, groups=1, top_groups=None, renormalize=True, scale=1.0):
    """(ids, weights) of one token, 64 bits."""
    l = [float(v) for v in logits]
    wrong = any(math.isnan(v) or (score == "softmax" and v == math.inf) for v in l) \
        or (bias is not None and any(math.isnan(float(b)) for b in bias))
    if wrong:
        return list(range(top)), [math.nan] * top
    n = len(l)
    s = scores(l, score)
    key = [-math.inf if l[e] == -math.inf else s[e] + float(bias[e]) if bias is not None else s[e] for e in range(n)]
    allowed = [key[e] > -math.inf for e in range(n)]
    if groups > 1:
        size = n // groups
        gs = []
        for g in range(groups):
            best = sorted((key[e] for e in range(g * size, (g + 1) * size) if allowed[e]), reverse=True)[:2]
            gs.append(sum(best) if best else -math.inf)
        keep = sorted(range(groups), key=lambda g: (-gs[g], g))[:top_groups or groups]
        allowed = [allowed[e] and e // size in keep for e in range(n)]
    rank = key if bias is not None else l
    ids = sorted((e for e in range(n) if allowed[e]), key=lambda e: (-rank[e], e))[:top]
    w = [s[e] for e in ids]
    if renormalize:
        if score == "softmax" and ids:   # relative to the chosen ones' highest, which may be far below the row's
            high = max(l[e] for e in ids)
            w = [math.exp(l[e] - high) for e in ids]
        total = math.fsum(w)
        w = [v / total if total > 0 else 0.0 for v in w]
    pad = top - len(ids)
    return ids + [-1] * pad, [scale * v for v in w] + [0.0] * pad


def route(logits, top, **how):
    out = [route_token(row, top, **how) for row in np.asarray(logits, dtype=np.float64)]
    return (np.array([o[0] for o in out], np.int32).reshape(-1, top), np.array([o[1] for o in out], np.float64).reshape(-1, top))


def weights_at(logits, ids, score="softmax", renormalize=True, scale=1.0):
    """The weights of given choices as a function of the logits (for differences)."""
    l = np.asarray(logits, dtype=np.float64)
    out = np.zeros(np.asarray(ids).shape)
    for t in range(len(l)):
        s = scores(l[t], score)
        w = [s[e] if e >= 0 else 0.0 for e in ids[t]]
        total = math.fsum(w)
        out[t] = [scale * (v / total if renormalize and total > 0 else v) for v in w]
    return out


def route_backward(logits, ids, dweights, score="softmax", renormalize=True, scale=1.0):
    """dL/dlogits [T, E] by the chain rule through every score, 64 bits."""
    l = np.asarray(logits, dtype=np.float64)
    out = np.zeros_like(l)
    for t in range(len(l)):
        s = np.array(scores(l[t], score))
        at = [int(e) for e in ids[t] if e >= 0]
        d = scale * np.array([float(dweights[t][j]) for j in range(len(ids[t])) if ids[t][j] >= 0])
        ds = np.zeros_like(s)
        if renormalize and at:
            total = math.fsum(s[at])
            if total > 0:
                ds[at] = (d - (d * s[at]).sum() / total) / total
        elif at:
            ds[at] = d
        if score == "softmax":
            out[t] = s * (ds - (s * ds).sum())
        else:
            one_minus = np.array(scores(-l[t], score))
            out[t] = ds * s * np.where(l[t] == -np.inf, 0.0, one_minus)
    return out


def group(ids, n):
    """(offsets, rows, slots) of choices ids [T, top] by expert 0 .. n - 1; rows only as far as they are owned."""
    ids = np.asarray(ids)
    top = ids.shape[1]
    lists = [[] for _ in range(n)]
    for i, e in enumerate(ids.reshape(-1)):
        if 0 <= e < n:
            lists[e].append(i)
    order = [i for one in lists for i in one]
    offsets = np.concatenate([[0], np.cumsum([len(one) for one in lists])]).astype(np.int32)
    slots = np.full(ids.size, -1, np.int32)
    slots[order] = np.arange(len(order))
    return offsets, (np.array(order, dtype=np.int64) // top).astype(np.int32), slots.reshape(ids.shape)
