"""Plain fp64 restatement of the node-level operators around a convolution:
type embedding, block norm (with gate and residual) and the gradient norm with
clipping.  Test infrastructure: shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def embedding(ids, table, scale=1.0):
    """y[i] = scale * table[ids[i]]; rows of out-of-range ids are 0."""
    ids, table = np.asarray(ids).reshape(-1).astype(np.int64), np.asarray(table, np.float64)
    y = np.zeros((len(ids), table.shape[1]))
    for i, v in enumerate(ids):
        if 0 <= v < len(table):
            y[i] = scale * table[v]
    return y


def embedding_grad(ids, gy, n_types, scale=1.0, padding=None):
    """dtable[v] = scale * sum of gy over the nodes of type v."""
    ids = np.asarray(ids).reshape(-1).astype(np.int64)
    gy = np.asarray(gy, np.float64).reshape(len(ids), -1)
    d = np.zeros((n_types, gy.shape[1]))
    for i, v in enumerate(ids):
        if 0 <= v < n_types and v != padding:
            d[v] += gy[i]
    return scale * d


def gate_function(kind, g):
    g = np.asarray(g, np.float64)
    s = 0.5 * (1.0 + np.tanh(0.5 * g))
    return {"none": np.ones_like(g), "sigmoid": s, "silu": g * s, "tanh": np.tanh(g)}[kind]


def gate_derivative(kind, g):
    g = np.asarray(g, np.float64)
    s = 0.5 * (1.0 + np.tanh(0.5 * g))
    return {"none": np.zeros_like(g), "sigmoid": s * (1 - s), "silu": s + g * s * (1 - s),
            "tanh": 1 - np.tanh(g) ** 2}[kind]


def _blocks(L):
    return [(l, slice(l * l, (l + 1) ** 2)) for l in range(L + 1)]


def block_norm(x, b, gate, w_post, w_pre, scale, eps, kind):
    """(x_out, h); None where not computed."""
    x = np.asarray(x, np.float64)
    L = int(round(x.shape[1] ** 0.5)) - 1
    y = x.copy()
    h = None if w_pre is None else np.empty_like(x)
    for l, rows in _blocks(L):
        if b is not None:
            v = np.asarray(b, np.float64)[:, rows]
            u = v / np.sqrt((v ** 2).mean(axis=(1, 2), keepdims=True) + eps) * np.asarray(w_post, np.float64)[l]
            a = 1.0 if kind == "none" else gate_function(kind, gate)[:, l][:, None]
            y[:, rows] += scale * a * u
        if w_pre is not None:
            v = y[:, rows]
            h[:, rows] = v / np.sqrt((v ** 2).mean(axis=(1, 2), keepdims=True) + eps) * np.asarray(w_pre, np.float64)[l]
    return (None if b is None else y), h


def block_norm_grad(x, b, gate, w_post, w_pre, g_x, g_h, scale, eps, kind):
    """(dx, db, dgate, dw_post, dw_pre) of <g_x, x_out> + <g_h, h>."""
    x = np.asarray(x, np.float64)
    L = int(round(x.shape[1] ** 0.5)) - 1
    C = x.shape[2]
    y = block_norm(x, b, gate, w_post, None, scale, eps, kind)[0] if b is not None else x
    t = np.zeros_like(x) if g_x is None else np.asarray(g_x, np.float64).copy()
    dwi = None if w_pre is None else np.zeros((L + 1, C))
    dwo = None if b is None else np.zeros((L + 1, C))
    db = None if b is None else np.zeros_like(x)
    dg = None if b is None or kind == "none" else np.zeros((x.shape[0], L + 1, C))
    for l, rows in _blocks(L):
        if g_h is not None:
            v, g = y[:, rows], np.asarray(g_h, np.float64)[:, rows]
            s = 1 / np.sqrt((v ** 2).mean(axis=(1, 2), keepdims=True) + eps)
            dwi[l] = (g * v * s).sum(axis=(0, 1))
            p = g * np.asarray(w_pre, np.float64)[l]
            t[:, rows] += s * p - v * s ** 3 * (p * v).mean(axis=(1, 2), keepdims=True)
        if b is not None:
            v = np.asarray(b, np.float64)[:, rows]
            s = 1 / np.sqrt((v ** 2).mean(axis=(1, 2), keepdims=True) + eps)
            a = np.ones((len(x), 1, C)) if kind == "none" else gate_function(kind, gate)[:, l][:, None]
            w = np.asarray(w_post, np.float64)[l]
            dwo[l] = (scale * a * t[:, rows] * v * s).sum(axis=(0, 1))
            if dg is not None:
                dg[:, l] = scale * gate_derivative(kind, gate)[:, l] * (t[:, rows] * v * s * w).sum(axis=1)
            q = scale * a * t[:, rows] * w
            db[:, rows] = s * q - v * s ** 3 * (q * v).mean(axis=(1, 2), keepdims=True)
    return t, db, dg, dwo, dwi


def gradient_norm(tensors):
    return float(np.sqrt(sum((np.asarray(t, np.float64) ** 2).sum() for t in tensors)))


def clip(tensors, max_norm, eps=1e-6):
    n = gradient_norm(tensors)
    with np.errstate(invalid="ignore"):
        k = np.minimum(1.0, np.float64(max_norm) / (n + eps))
        return n, [np.asarray(t, np.float64) * k for t in tensors]
