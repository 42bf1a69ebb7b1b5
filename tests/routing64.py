"""Routing and row moving in numpy's 64-bit types, for the checks of the kernels: written from the definitions, token by
token and row by row, without the library."""
import numpy as np


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def scores(l, score):
    """p [tokens, experts] in 64 bits; rows of -inf alone give zeros"""
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(l == -np.inf, 0.0, sigmoid(l))
    top = l.max(1, keepdims=True)
    e = np.exp(l - np.where(np.isfinite(top), top, 0.0))
    s = e.sum(1, keepdims=True)
    return e / np.where(s > 0, s, 1.0)


def choices(l32, bias32, k):
    """int [tokens, k]: the experts of the k largest float32 sums above -inf, ties to the lowest, -1 for none"""
    c = l32 if bias32 is None else (l32 + bias32).astype(np.float32)
    c = np.where(np.isnan(c), np.float32(np.inf), c).astype(np.float64) + np.where(np.isnan(c), 1e300, 0.0)
    e = np.argsort(-c, axis=1, kind="stable")[:, :k]
    return np.where(np.take_along_axis(c, e, 1) == -np.inf, -1, e)


def gates(l, chosen, score, normalize, scale=1.0):
    p = scores(l, score)
    at = np.maximum(chosen, 0)
    g = np.where(chosen >= 0, np.take_along_axis(p, at, 1), 0.0)
    if normalize:
        v = np.take_along_axis(l, at, 1)
        v = v if score == "softmax" else np.minimum(v, 0) - np.log1p(np.exp(-np.abs(v)))  # log p
        v = np.where(chosen >= 0, v, -np.inf)
        top = v.max(1, keepdims=True)
        e = np.exp(v - np.where(np.isfinite(top), top, 0.0))
        s = e.sum(1, keepdims=True)
        g = e / np.where(s > 0, s, 1.0)
    return scale * g


def gates_backward(l, chosen, d, score, normalize, scale=1.0):
    """dlogits, and the sum of the magnitudes of the terms that make each of them"""
    q = gates(l, chosen, score, normalize)
    d = np.where(chosen >= 0, d, 0.0)
    dl, mag = np.zeros((2,) + l.shape)
    p = scores(l, score)
    for t in range(l.shape[0]):
        dot, adot = (q[t] * d[t]).sum(), np.abs(q[t] * d[t]).sum()
        if score == "softmax" and not normalize:
            dl[t], mag[t] = -scale * p[t] * dot, abs(scale) * p[t] * adot
        for i, e in enumerate(chosen[t]):
            if e < 0:
                continue
            if score == "softmax":
                dl[t, e], mag[t, e] = scale * q[t, i] * (d[t, i] - dot), q[t, i] * (abs(d[t, i]) + adot)
            elif normalize:
                dl[t, e] = scale * q[t, i] * (d[t, i] - dot) * (1 - p[t, e])
                mag[t, e] = q[t, i] * (abs(d[t, i]) + adot) * (1 - p[t, e])
            else:
                dl[t, e] = scale * p[t, e] * (1 - p[t, e]) * d[t, i]
                mag[t, e] = abs(dl[t, e])
    return dl, np.abs(mag) * max(1.0, abs(scale))


def layout(chosen, experts, pad, rows):
    """(offsets, row_index, row_choice)"""
    counts = [(chosen == e).sum() for e in range(experts)]
    offsets = np.concatenate([[0], np.cumsum([-(-c // pad) * pad for c in counts])]).astype(np.int64)
    index, choice = np.full(chosen.size, -1), np.full(rows, -2)
    choice[:offsets[-1]] = -1
    for e in range(experts):
        mine = np.flatnonzero(chosen.reshape(-1) == e)
        choice[offsets[e]:offsets[e] + len(mine)] = mine
        index[mine] = offsets[e] + np.arange(len(mine))
    return offsets, index.reshape(chosen.shape), choice
