"""Float64 definitions of what stands in front of a routed layer and keeps its
backward pass small: rows held in 8 bits, the root-mean-square norm, routing
from scores, each with its gradient.

Plain numpy and Python loops, following the definitions term by term; shares no
code with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------------------ rows in 8 bits
def scale_exponent(m, fmt):
    """Least e from -126 on with m < 127.5 2^e ("int8") or m <= 464 2^e ("e4m3")."""
    e = -126
    if fmt == "int8":
        while not m < math.ldexp(127.5, e):
            e += 1
    else:
        while not m <= math.ldexp(464.0, e):
            e += 1
    return e


def e4m3_values():
    """Every non-negative value of the type, ascending: code c has value e4m3_values()[c]."""
    out = []
    for c in range(0x7f):
        exp, man = c >> 3, c & 7
        out.append(man * 2.0 ** -9 if exp == 0 else (8 + man) * 2.0 ** (exp - 10))
    return out


def round_e4m3(q):
    """Nearest value of the type, ties to the even code."""
    vals = e4m3_values()
    a = abs(q)
    best = min(range(len(vals)), key=lambda c: (abs(vals[c] - a), c & 1))
    return math.copysign(vals[best], q)


def eight(v, fmt, block):
    """(values, scales) of the 8-bit rows of v [M, N]."""
    M, N = v.shape
    B = -(-N // block)
    out, scales = np.zeros((M, N)), np.ones((M, B))
    for i in range(M):
        for b in range(B):
            part = v[i, b * block:(b + 1) * block]
            if not np.isfinite(part).all():
                scales[i, b] = math.nan
                out[i, b * block:(b + 1) * block] = math.nan
                continue
            m = float(np.abs(part).max())
            s = 1.0 if m == 0.0 else math.ldexp(1.0, scale_exponent(m, fmt))
            scales[i, b] = s
            for j, x in enumerate(part):
                q = float(x) / s
                out[i, b * block + j] = (round(q) if fmt == "int8" else round_e4m3(q)) * s
    return out, scales


def values(codes, scales, fmt, block):
    """What codes (uint8 as stored) and scales stand for."""
    if fmt == "int8":
        table = np.arange(256) - 128.0
    else:
        half = np.array(e4m3_values() + [math.nan])
        table = np.concatenate([half, -half])
    return table[codes] * np.repeat(scales, block, axis=1)[:, :codes.shape[1]]


def slots(rows, perm, k):
    """Row perm[m] / k for every m; zeros where perm lies outside the slots."""
    out = np.zeros((len(perm), rows.shape[1]))
    for m, p in enumerate(perm):
        if 0 <= p < len(perm):
            out[m] = rows[p // k]
    return out


# ------------------------------------------------------------------ norm
def rms_norm(h, w=None, eps=1e-6):
    out = np.zeros(h.shape)
    for i, row in enumerate(h):
        s = 1.0 / math.sqrt(math.fsum(float(v) * float(v) for v in row) / len(row) + eps)
        out[i] = row * s
    return out if w is None else out * w


def rms_norm_grad(dy, h, w=None, ds=None, eps=1e-6):
    """(grad_input, grad_weight)."""
    M, H = h.shape
    dh, dw = np.zeros((M, H)), np.zeros(H)
    one = np.ones(H) if w is None else w
    for i in range(M):
        ms = math.fsum(float(v) * float(v) for v in h[i]) / H + eps
        s = 1.0 / math.sqrt(ms)
        g = dy[i] * one
        # d y_j / d h_c = w_j (s [j = c] - h_j h_c / (H ms^(3/2)))
        dh[i] = g * s - h[i] * (math.fsum(g * h[i]) / (H * ms * math.sqrt(ms)))
        dw += dy[i] * h[i] * s
    if ds is not None:
        dh = dh + ds
    return dh, dw


# ------------------------------------------------------------------ routing from scores
BIGGEST = float(np.finfo(np.float32).max)


def scores(logits, kind):
    """[T, E] scores and which experts are masked; a logit of +infinity counts as the largest float."""
    T, E = logits.shape
    off = np.isnan(logits) | (logits == -np.inf)
    s = np.zeros((T, E))
    for t in range(T):
        l = [min(float(v), BIGGEST) for v in logits[t]]
        on = [e for e in range(E) if not off[t, e]]
        if kind == "sigmoid":
            for e in on:
                s[t, e] = 1.0 / (1.0 + math.exp(-l[e])) if l[e] > -700 else math.exp(max(l[e], -740.0))
        elif on:
            top = max(l[e] for e in on)
            ex = {e: math.exp(max(l[e] - top, -745.0)) if l[e] - top > -745.0 else 0.0 for e in on}
            total = math.fsum(ex.values())
            for e in on:
                s[t, e] = ex[e] / total
    return s, off


def route_scored(logits, k, kind="softmax", bias=None, groups=1, kept=1, group_top=2, normalize=0, scale=1.0):
    """(indices, weights): a token at a time.  Scores, scores plus bias and sums of two count as float32 where experts
    and groups are ranked."""
    T, E = logits.shape
    s, off = scores(logits, kind)
    s32 = s.astype(np.float32)
    per = E // groups
    idx, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        c = {}
        for e in range(E):
            if off[t, e]:
                continue
            v = s32[t, e] if bias is None else np.float32(s32[t, e] + np.float32(bias[e]))
            if not np.isnan(v) and v != -np.inf:
                c[e] = float(v)
        rank = []
        for g in range(groups):
            best = sorted((c[e] for e in c if e // per == g), reverse=True)[:group_top]
            rank.append(float(np.float32(sum(best))) if best else -math.inf)
        keep = sorted(range(groups), key=lambda g: (-rank[g], g))[:kept]
        pick = sorted((e for e in c if e // per in keep), key=lambda e: (-c[e], e))[:k]
        total = math.fsum(float(s32[t, e]) for e in pick)
        for i, e in enumerate(pick):
            idx[t, i] = e
            v = float(s32[t, e])
            w[t, i] = scale * (v if not normalize else v / total if total > 0 else 0.0)
    return idx, w


def route_scored_grad(grad_w, logits, idx, kind="softmax", normalize=0, scale=1.0):
    """Gradient at the logits, the selection constant, by the chain rule through the scores (as rounded to float32; the
    library does not round them here)."""
    T, E = logits.shape
    s, off = scores(logits, kind)
    s = s.astype(np.float32).astype(np.float64)
    out = np.zeros((T, E))
    for t in range(T):
        sel = [(i, int(e)) for i, e in enumerate(idx[t]) if 0 <= e < E and not off[t, int(e)]]
        g = {i: scale * float(grad_w[t, i]) for i, _ in sel}
        ds = np.zeros(E)
        if normalize:
            total = math.fsum(s[t, e] for _, e in sel)
            if total > 0:
                mean = math.fsum(g[i] * s[t, e] for i, e in sel) / total
                for i, e in sel:
                    ds[e] += (g[i] - mean) / total
        else:
            for i, e in sel:
                ds[e] += g[i]
        if kind == "sigmoid":
            for e in range(E):
                if not off[t, e]:
                    l = min(float(logits[t, e]), BIGGEST)
                    out[t, e] = ds[e] * s[t, e] * (1.0 / (1.0 + math.exp(l)) if l < 700 else 0.0)
        else:
            mean = math.fsum(ds * s[t])
            out[t] = s[t] * (ds - mean)
    return out
