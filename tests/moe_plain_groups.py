"""Plain 64-bit form of the router by groups (CPU, numpy loops), written from the
definition in include/a2av_moe.h."""
from __future__ import annotations

import math

import numpy as np


def scores(l, kind: str):
    with np.errstate(invalid="ignore", over="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-l))
        free = l != -math.inf
        if not free.any():
            return np.zeros_like(l)
        p = np.where(free, np.exp(l - np.nanmax(np.where(free, l, -math.inf))), 0.0)
        return p / p.sum()


def rank(values, among):
    """The numbers of `among`, NaN first, then by falling value, equal ones by number."""
    return sorted(among, key=lambda i: (0, 0.0, i) if math.isnan(values[i]) else (1, -values[i], i))


def route(logits, k, kind, bias, groups, top_groups, best, renorm, scale):
    """experts, weights, counts, order, place of the definition, in float64."""
    T, E = logits.shape
    size = E // groups
    experts = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k))
    for t in range(T):
        l = logits[t].astype(np.float64)
        s = scores(l, kind)
        c = s if bias is None else s + bias.astype(np.float64)
        free = [e for e in range(E) if l[e] != -math.inf and c[e] != -math.inf]
        of_group = {}
        for g in range(groups):
            mine = rank(c, [e for e in free if e // size == g])[:best]
            if mine:
                of_group[g] = sum(c[e] for e in mine)
        taken = rank(of_group, of_group)[:top_groups]
        chosen = rank(l if bias is None else c, [e for e in free if e // size in taken])[:k]
        experts[t, :len(chosen)] = chosen
        if chosen:
            total = s[chosen].sum() if renorm else 1.0
            weights[t, :len(chosen)] = scale * s[chosen] / total if total != 0 else 0.0
    counts = np.bincount(experts[experts >= 0], minlength=E).astype(np.int32)
    order = np.full(T * k, -1, np.int32)
    place = np.full(T * k, -1, np.int32)
    flat = experts.reshape(-1)
    slots = np.argsort(np.where(flat < 0, E, flat), kind="stable")
    n = int((flat >= 0).sum())
    order[:n] = slots[:n] // k
    place[slots[:n]] = np.arange(n)
    return experts, weights, counts, order, place.reshape(T, k)


def route_back(logits, experts, dweights, kind, renorm, scale):
    """By the chain rule through the scores, from the scores in float64."""
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        l = logits[t].astype(np.float64)
        s = scores(l, kind)
        at = [e for e in experts[t] if e >= 0]
        g = dweights[t][[j for j, e in enumerate(experts[t]) if e >= 0]].astype(np.float64)
        ds = np.zeros(E)
        total = s[at].sum() if renorm else 1.0
        if at and total > 0:
            ds[at] = scale / total * (g - (s[at] / total @ g if renorm else 0.0))
        if kind == "sigmoid":
            out[t] = ds * s * (1 / (1 + np.exp(l)))
        else:
            out[t] = s * (ds - s @ ds)
    return out
