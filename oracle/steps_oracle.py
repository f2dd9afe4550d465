"""Float64 definitions of the steps of a routed layer and their gradients:
routing weights, token dispatch and combine, linear layers.

Plain numpy loops and dot products, following the definitions term by term;
shares no code with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------------------ routing weights
def route(logits, k, routing="qmoe", normalize=0):
    """(indices, weights) of logits [T, E]: a token at a time."""
    T, E = logits.shape
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        row = [float(v) for v in logits[t]]
        left = [e for e in range(E) if not math.isnan(row[e]) and row[e] != -math.inf]
        left.sort(key=lambda e: (-row[e], e))
        pick = left[:k]
        over = left if routing == "moe" and not normalize else pick
        total = sum(math.exp(row[e] - row[left[0]]) for e in over)
        for s, e in enumerate(pick):
            idx[t, s] = e
            w[t, s] = math.exp(row[e] - row[left[0]]) / total
    return idx, w


def route_grad(grad_w, logits, idx, routing="qmoe", normalize=0):
    """Gradient at the logits, the selection constant: the softmax's Jacobian
    row by row."""
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        row = logits[t].astype(np.float64)
        usable = [e for e in range(E) if not math.isnan(row[e]) and row[e] != -math.inf]
        slots = [(s, int(e)) for s, e in enumerate(idx[t]) if 0 <= e < E and int(e) in usable]
        over = usable if routing == "moe" and not normalize else [e for _, e in slots]
        if not over:
            continue
        top = max(row[e] for e in over)
        total = sum(math.exp(row[e] - top) for e in over)
        for s, e in slots:
            p = math.exp(row[e] - top) / total
            for f in over:  # d p_e / d l_f = p_e ([e = f] - p_f), one term per member of the sum
                out[t, f] -= grad_w[t, s] * p * math.exp(row[f] - top) / total
            out[t, e] += grad_w[t, s] * p
    return out


# ------------------------------------------------------------------ dispatch and combine
def sort_slots(idx, experts):
    """(offsets, perm, inverse) of indices [T, k]: slots listed expert by expert, then the dropped ones."""
    T, k = idx.shape
    order, offsets = [], [0]
    flat = idx.reshape(-1)
    for e in range(experts):
        order += [s for s in range(T * k) if flat[s] == e]
        offsets.append(len(order))
    order += [s for s in range(T * k) if not 0 <= flat[s] < experts]
    inverse = np.zeros(T * k, np.int32)
    for p, s in enumerate(order):
        inverse[s] = p if p < offsets[-1] else -1 - p
    return np.array(offsets, np.int32), np.array(order, np.int32).reshape(-1), inverse.reshape(T, k)


def dispatch(x, idx, experts):
    offsets, perm, inverse = sort_slots(idx, experts)
    k = idx.shape[1]
    rows = np.zeros((idx.size, x.shape[1]), x.dtype)
    for p in range(offsets[-1]):
        rows[p] = x[perm[p] // k]
    return rows, offsets, perm, inverse


def combine(rows, inverse, weights=None):
    T, k = inverse.shape
    out = np.zeros((T, rows.shape[1]))
    for t in range(T):
        for s in range(k):
            if 0 <= inverse[t, s] < T * k:
                out[t] += (1.0 if weights is None else float(weights[t, s])) * rows[inverse[t, s]].astype(np.float64)
    return out


def combine_grad(grad_out, rows, inverse, weights):
    T, k = inverse.shape
    gr, gw = np.zeros(rows.shape), np.zeros((T, k))
    for t in range(T):
        for s in range(k):
            if inverse[t, s] >= 0:
                gr[inverse[t, s]] = float(weights[t, s]) * grad_out[t].astype(np.float64)
                gw[t, s] = grad_out[t].astype(np.float64) @ rows[inverse[t, s]].astype(np.float64)
    return gr, gw


# ------------------------------------------------------------------ linear layers
def _phi(z):
    return np.vectorize(lambda v: 0.5 * math.erfc(-v / math.sqrt(2.0)), otypes=[np.float64])(z)


def _sigma(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def act(z, kind, alpha=1.0, beta=0.0, limit=None):
    if kind == "identity":
        return z.copy()
    if kind == "relu":
        return np.where(z < 0, 0.0, z)
    if kind == "gelu":
        return z * _phi(z)
    if kind == "silu":
        return z * _sigma(z)
    g, u = z[:, 0::2], z[:, 1::2]
    if limit is not None:
        g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
    return g * _sigma(alpha * g) * (u + beta)


def act_grad(dy, z, kind, alpha=1.0, beta=0.0, limit=None):
    """Gradient at z [M, N] of act's output."""
    if kind == "identity":
        return dy.copy()
    if kind == "relu":
        return np.where(z > 0, dy, 0.0)
    if kind == "gelu":
        return dy * (_phi(z) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    if kind == "silu":
        s = _sigma(z)
        return dy * (s + z * s * (1 - s))
    g, u = z[:, 0::2], z[:, 1::2]
    gp, up = np.ones(g.shape), np.ones(u.shape)
    if limit is not None:
        gp, up = (g <= limit) * 1.0, (np.abs(u) <= limit) * 1.0
        g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
    s = _sigma(alpha * g)
    out = np.zeros(z.shape)
    out[:, 0::2] = dy * (u + beta) * (s + alpha * g * s * (1 - s)) * gp
    out[:, 1::2] = dy * g * s * up
    return out


def spans(M, G, offsets):
    if offsets is None:
        return [(0, M)]
    return [(int(offsets[g]), int(offsets[g + 1])) for g in range(G)]


def preact(x, w, b, offsets=None):
    """z [M, N]; rows behind the last group zero.  w [N, K] or [G, N, K]."""
    M = x.shape[0]
    w3 = w if w.ndim == 3 else w[None]
    b2 = None if b is None else b.reshape(w3.shape[:2])
    z = np.zeros((M, w3.shape[1]))
    for g, (lo, hi) in enumerate(spans(M, w3.shape[0], offsets)):
        z[lo:hi] = x[lo:hi] @ w3[g].T
        if b2 is not None:
            z[lo:hi] += b2[g]
    return z


def live_rows(M, w, offsets):
    return M if offsets is None else int(offsets[w.shape[0]])


def linear(x, w, b=None, r=None, offsets=None, kind="identity", **a):
    """(output, preact)."""
    z = preact(x, w, b, offsets)
    n = live_rows(x.shape[0], w, offsets)
    y = act(z, kind, **a)
    if r is not None:
        y[:n] += r[:n]
    y[n:] = 0.0
    return y, z


def linear_grad(dy, x, w, z=None, offsets=None, kind="identity", **a):
    """(grad_input, grad_weights, grad_bias, d)."""
    M = x.shape[0]
    w3 = w if w.ndim == 3 else w[None]
    d = act_grad(dy, z, kind, **a)
    dx, dw, db = np.zeros(x.shape), np.zeros(w3.shape), np.zeros(w3.shape[:2])
    for g, (lo, hi) in enumerate(spans(M, w3.shape[0], offsets)):
        dx[lo:hi] = d[lo:hi] @ w3[g]
        dw[g] = d[lo:hi].T @ x[lo:hi]
        db[g] = d[lo:hi].sum(0)
    return dx, dw.reshape(w.shape), db.reshape(w.shape[:-1]), d
