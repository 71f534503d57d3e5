"""Plain 64-bit implementation of what surrounds a mixture's products, on numpy arrays: routing with
its balance loss and gradients, a product's epilogue, the sum of the experts' rows and its gradients.

Independent of the package, and written from the definitions, row by row.
"""
from __future__ import annotations

import numpy as np


def route(logits, top: int, normalize: bool):
    """dict of weight, expert, slot [rows, top], index [rows * top], offsets, counts, loss and p."""
    x = np.asarray(logits, np.float64)
    rows, experts = x.shape
    weight, expert = np.zeros((rows, top)), np.full((rows, top), -1)
    p = np.zeros((rows, experts))
    used = 0
    for t in range(rows):
        row = x[t]
        if np.isnan(row).any() or (row == np.inf).any():
            weight[t], p[t] = np.nan, np.nan
            used += 1
            continue
        open_ = row > -np.inf
        if not open_.any():
            continue
        used += 1
        m = row.max()
        e = np.where(open_, np.exp(np.where(open_, row, m) - m), 0.0)
        p[t] = e / e.sum()
        order = [i for i in np.argsort(-row, kind="stable") if open_[i]][:top]
        expert[t, :len(order)] = order
        weight[t, :len(order)] = e[order] / e[order].sum() if normalize else p[t, order]
    slot, index = np.full((rows, top), -1), np.full(rows * top, -1)
    counts, offsets = np.zeros(experts + 2, int), np.zeros(experts + 1, int)
    next_ = 0
    for e in range(experts):
        offsets[e] = next_
        for t, j in zip(*np.nonzero(expert == e)):
            slot[t, j], index[next_] = next_, t
            next_ += 1
        counts[e] = next_ - offsets[e]
    offsets[experts] = counts[experts] = next_
    counts[experts + 1] = used
    with np.errstate(invalid="ignore"):
        loss = experts * float((counts[:experts] / max(next_, 1) * p.sum(0) / max(used, 1)).sum())
    return dict(weight=weight, expert=expert, slot=slot, index=index, offsets=offsets, counts=counts, loss=loss, p=p)


def route_objective(logits, expert, counts, dweight, dloss, normalize: bool) -> float:
    """sum w dw + dloss L as a function of the logits, the choices and counts being what they are."""
    x = np.asarray(logits, np.float64)
    experts = x.shape[1]
    total, mean = 0.0, np.zeros(experts)
    for t, row in enumerate(x):
        if not (row > -np.inf).any():
            continue
        e = np.exp(row - row.max())
        mean += e / e.sum()
        c = expert[t][expert[t] >= 0]
        w = e[c] / (e[c].sum() if normalize else e.sum())
        total += float(w @ np.asarray(dweight, np.float64)[t, :len(c)])
    made, used = max(int(counts[experts]), 1), max(int(counts[experts + 1]), 1)
    return total + float(dloss) * experts * float((counts[:experts] / made * mean / used).sum())


def route_backward(r: dict, dweight, dloss, normalize: bool):
    """The gradient of route_objective, from route's results."""
    p, rows, experts = r["p"], *r["p"].shape
    made, used = max(int(r["counts"][experts]), 1), max(int(r["counts"][experts + 1]), 1)
    b = float(dloss) * experts * r["counts"][:experts] / (made * used)
    dl = p * (b - (p * b).sum(1, keepdims=True))
    for t in range(rows):
        c = r["expert"][t]
        k = int((c >= 0).sum())
        w, g = r["weight"][t, :k], np.asarray(dweight, np.float64)[t, :k]
        if normalize:
            dl[t, c[:k]] += w * (g - w @ g)
        else:
            dl[t] -= p[t] * (w @ g)
            dl[t, c[:k]] += w * g
    return dl


def combine(z, slot, weight=None, residual=None):
    z = np.asarray(z, np.float64)
    rows, top = slot.shape
    y = np.zeros((rows, z.shape[1])) if residual is None else np.array(residual, np.float64)
    for t in range(rows):
        for j in range(top):
            w = 1.0 if weight is None else float(weight[t, j])
            s = int(slot[t, j])
            y[t] += w * z[s] if 0 <= s < z.shape[0] else w * 0.0
    return y


def combine_backward(dy, z, slot, weight=None):
    """(dz with NaN in rows that no choice names, dweight)."""
    dy, z = np.asarray(dy, np.float64), np.asarray(z, np.float64)
    dz, dw = np.full(z.shape, np.nan), np.zeros(slot.shape)
    for t in range(slot.shape[0]):
        for j in range(slot.shape[1]):
            s = int(slot[t, j])
            if 0 <= s < z.shape[0]:
                dz[s] = dy[t] * (1.0 if weight is None else float(weight[t, j]))
                dw[t, j] = dy[t] @ z[s]
    return dz, dw


def activation(v, act: str):
    v = np.asarray(v, np.float64)
    if act == "relu":
        return np.where(v < 0, 0.0, v)
    if act == "silu":
        with np.errstate(over="ignore"):
            return v / (1 + np.exp(-v))
    if act == "gelu":
        from scipy.special import ndtr
        return v * ndtr(v)
    if act == "gelu_tanh":
        return 0.5 * v * (1 + np.tanh(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))
    return v
