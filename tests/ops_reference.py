"""Plain 64-bit forms (numpy) of the router, its gradient, the combine's
gradient and the experts' products with 4-bit weights, written from their
definitions for the tests."""
from __future__ import annotations

import numpy as np


def scores(logits: np.ndarray, kind: str) -> np.ndarray:
    l = logits.astype(np.float64)
    on = l > -np.inf  # false for NaN
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(on, 1.0 / (1.0 + np.exp(-np.where(on, l, 0.0))), 0.0)
    top = np.max(np.where(on, l, -np.inf), axis=1, keepdims=True)
    e = np.zeros_like(l)
    for t in range(l.shape[0]):
        m = top[t, 0]
        if m == np.inf:
            e[t] = on[t] & (l[t] == np.inf)
        elif m > -np.inf:
            e[t, on[t]] = np.exp(l[t, on[t]] - m)
    s = e.sum(1, keepdims=True)
    return np.where(s > 0, e / np.where(s > 0, s, 1.0), 0.0)


def route_keys(logits, kind, bias=None):
    """Keys of the choice (-inf: not to be chosen)."""
    l = logits.astype(np.float64)
    key = scores(logits, kind) if (kind == "sigmoid" or bias is not None) else l.copy()
    if bias is not None:
        key = key + bias.astype(np.float64)
    return np.where(l > -np.inf, key, -np.inf)


def keep_groups(key, kind, num_groups, topk_groups):
    T, E = key.shape
    parts = np.sort(key.reshape(T, num_groups, -1), axis=2)[..., ::-1]
    g = parts[..., 0].copy()
    if kind == "sigmoid" and parts.shape[2] > 1:
        second = parts[..., 1]
        g = g + np.where(second > -np.inf, second, 0.0)
    order = np.argsort(-g, axis=1, kind="stable")[:, :topk_groups]
    kept = np.zeros((T, num_groups), bool)
    np.put_along_axis(kept, order, True, axis=1)
    return np.where(np.repeat(kept, E // num_groups, axis=1), key, -np.inf), g


def choose(key, K):
    idx = np.argsort(-key, axis=1, kind="stable")[:, :K]
    return np.where(np.take_along_axis(key, idx, 1) > -np.inf, idx, -1)


def route_weights(logits, idx, kind, renorm, scale):
    s = scores(logits, kind)
    u = np.where(idx >= 0, np.take_along_axis(s, np.maximum(idx, 0), 1), 0.0)
    if renorm:
        if kind == "softmax":  # the softmax over the chosen logits
            l = np.where(idx >= 0, np.take_along_axis(logits.astype(np.float64),
                                                      np.maximum(idx, 0), 1), -np.inf)
            u = scores(l, "softmax")
        tot = u.sum(1, keepdims=True)
        u = np.where(tot > 0, u / np.where(tot > 0, tot, 1.0), 0.0)
    return u * scale


def route_grad(dw, logits, idx, kind, renorm, scale):
    """The gradient from the definition: through du and the scores."""
    T, E = logits.shape
    l = logits.astype(np.float64)
    s = scores(logits, kind)
    ok = (idx >= 0) & (idx < E)
    at = np.where(ok, idx, 0)
    ok &= np.take_along_axis(l, at, 1) > -np.inf
    u = np.where(ok, np.take_along_axis(s, at, 1), 0.0)
    d = np.where(ok, dw.astype(np.float64) * scale, 0.0)
    if renorm:
        S = u.sum(1, keepdims=True)
        r = np.where(S > 0, 1.0 / np.where(S > 0, S, 1.0), 0.0)
        d = (d - (d * u * r).sum(1, keepdims=True)) * r * ok
    ds = np.zeros_like(s)
    for k in range(idx.shape[1]):
        np.add.at(ds, (np.arange(T)[ok[:, k]], at[ok[:, k], k]), d[ok[:, k], k])
    if kind == "sigmoid":
        return ds * s * (1.0 - s)
    return s * (ds - (s * ds).sum(1, keepdims=True))


def dequantize_w4(q, scales, zeros):
    """[..., N, I/2] codes, [..., N, I/group] scales and zero points -> [..., N, I]."""
    I = 2 * q.shape[-1]
    group = I // scales.shape[-1]
    v = np.stack((q & 15, q >> 4), axis=-1).reshape(*q.shape[:-1], I).astype(np.float64)
    z = np.full(scales.shape, 8.0) if zeros is None else zeros.astype(np.float64)
    return (v - np.repeat(z, group, -1)) * np.repeat(scales.astype(np.float64), group, -1)


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))
