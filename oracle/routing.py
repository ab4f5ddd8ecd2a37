"""Expert routing definitions (test infrastructure only), in FP64 numpy.

Row t is live where valid[t] and some logit lies above -infinity. The choices
of a live row are its k largest logits (ties: lowest index; -infinity and NaN
are not chosen). loss = E / (k n) * sum_e counts[e] * mean_t p[t, e] over the n
live rows.
"""
from __future__ import annotations

import numpy as np


def route(logits, k: int, valid=None, normalize: bool = True) -> dict:
    """Everything a routing decides: ids, weights, counts, offsets, rows, pos,
    mean_probs, loss, n_valid, and the probabilities p [T, E] (0 in rows that
    are not live)."""
    x = np.asarray(logits, dtype=np.float64)
    t, e = x.shape
    mask = np.ones(t, bool) if valid is None else np.asarray(valid).astype(bool)
    p = np.zeros((t, e))
    ids = np.full((t, k), -1, np.int32)
    w = np.zeros((t, k))
    live = np.zeros(t, bool)
    with np.errstate(invalid="ignore"):
        for i in range(t):
            can = x[i] > -np.inf                       # False for NaN
            if not mask[i] or not can.any():
                continue
            live[i] = True
            z = np.exp(x[i] - x[i][can].max())
            p[i] = z / z.sum()
            order = sorted(np.nonzero(can)[0], key=lambda f: (-x[i, f], f))[:k]
            ids[i, : len(order)] = order
            w[i, : len(order)] = p[i, order] / (p[i, order].sum() if normalize else 1.0)
    n = int(live.sum())
    places = [[] for _ in range(e)]
    for i in range(t):
        for j in range(k):
            if ids[i, j] >= 0:
                places[ids[i, j]].append((i, j))
    counts = np.array([len(q) for q in places], np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = np.full(t * k, -1, np.int32)
    pos = np.full((t, k), -1, np.int32)
    at = 0
    for q in places:
        for i, j in q:
            rows[at] = i
            pos[i, j] = at
            at += 1
    mean = p.sum(0) / n if n else np.zeros(e)
    loss = e / (k * n) * float((counts * mean).sum()) if n else 0.0
    return {"ids": ids, "weights": w, "counts": counts, "offsets": offsets, "rows": rows, "pos": pos,
            "mean_probs": mean, "loss": loss, "n_valid": n, "p": p}


def route_backward(r: dict, k: int, normalize: bool = True, dweights=None, dloss=None):
    """(dlogits, scale): the gradient, and for every element the sum of the
    magnitudes of the terms that make it up (what rounding errors of a
    computation of it are measured against)."""
    p, ids, w = r["p"], r["ids"], r["weights"]
    t, e = p.shape
    n = r["n_valid"]
    c = np.zeros(e) if dloss is None or n == 0 else float(dloss) * e / (k * n * n) * r["counts"].astype(np.float64)
    d = p * (c - p @ c[:, None])
    mag = p * (np.abs(c) + p @ np.abs(c)[:, None])
    if dweights is not None:
        dw = np.where(ids >= 0, np.asarray(dweights, np.float64), 0.0)
        inner = (w * dw).sum(1, keepdims=True)
        size = (w * np.abs(dw)).sum(1, keepdims=True)
        for i in range(t):
            for j in range(k):
                if ids[i, j] < 0:
                    continue
                if normalize:
                    d[i, ids[i, j]] += w[i, j] * (dw[i, j] - inner[i, 0])
                    mag[i, ids[i, j]] += w[i, j] * (abs(dw[i, j]) + size[i, 0])
                else:
                    d[i, ids[i, j]] += w[i, j] * dw[i, j]
                    mag[i, ids[i, j]] += w[i, j] * abs(dw[i, j])
        if not normalize:
            d -= p * inner
            mag += p * size
    return d, mag
