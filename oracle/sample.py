"""Sampling of a token in fp64 (numpy): the definition of dsa_sample, one row at a time."""
from __future__ import annotations

import math

import numpy as np


def kept_tokens(x, temperature, top_k=0, top_p=1.0, min_p=0.0):
    """(kept tokens in ascending order, their weights, margin): margin is how near, as a part of the mass, top-p's
    border lies to a sum of weights."""
    x = np.asarray(x, dtype=np.float64)
    usable = np.flatnonzero(np.isfinite(x))
    if usable.size == 0:
        return usable, x[:0], math.inf
    order = usable[np.argsort(-x[usable], kind="stable")]
    if temperature == 0:
        return order[:1], np.ones(1), math.inf
    z = (x[order] - x[order[0]]) / temperature
    w = np.exp(z)
    n, margin = order.size, math.inf
    if min_p > 0:
        n = int((z >= math.log(min_p)).sum())
    if top_k > 0:
        n = min(n, top_k)
    if top_p < 1:
        before = np.cumsum(w[:n].astype(np.longdouble)) - w[:n]
        border = np.longdouble(top_p) * w[:n].sum(dtype=np.longdouble)
        margin = float(np.abs(before[1:] - border).min() / before[-1]) if n > 1 else math.inf
        n = max(1, int((before < border).sum()))
    kept = np.sort(order[:n])
    return kept, np.exp((x[kept] - x[order[0]]) / temperature), margin


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probability, margin): margin also of the draw."""
    kept, w, margin = kept_tokens(x, temperature, top_k, top_p, min_p)
    if kept.size == 0:
        return -1, 0.0, margin
    if temperature == 0:
        return int(kept[0]), 1.0, margin
    mass = np.cumsum(w.astype(np.longdouble))
    i = min(int((mass <= np.longdouble(u) * mass[-1]).sum()), kept.size - 1)
    margin = min(margin, float(np.abs(mass[:-1] / mass[-1] - np.longdouble(u)).min()) if kept.size > 1 else math.inf)
    return int(kept[i]), float(w[i] / mass[-1]), margin
