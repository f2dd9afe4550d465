"""GPU parity of the gradient of routing from scores where its sums cancel.

Renormalised, an expert's gradient is f_e times the sum over its slots of

    g_i - shift = sum_j w_j (g_i - g_j),   w = s / S,

which is 0 for a single slot and far below the g's where one slot holds nearly all of S; without renormalisation the
softmax's is s_e (D_e - sum_i s_i g_i) = s_e (D_e (1 - s_e) - the other slots' s_i g_i).  The references below are these
differences, which do not cancel where one slot dominates, in float64.

Bounds: scores are within 2^-44 of themselves (an exponential to 2^-50 of a float64 difference of at most 110, whose
rounding is 2^-47), sums and differences of k float64 terms of at most G = max |g| and the two products behind them
within (k + 16) 2^-44 G f, and one rounding to float32 follows (half a subnormal step at least)."""
import numpy as np
import pytest

import quantized_mixture_experts_router_amd as qm

import steps_util as U

pytestmark = pytest.mark.gpu

KINDS = ["softmax", "sigmoid"]


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.skip("no GPU")
    return _t


def scores_of(l, kind):
    """(s, 1 - s for the sigmoid, masked) of finite or -infinity / NaN logits."""
    off = np.isnan(l) | (l == -np.inf)
    l = np.where(off, -1e30, l)
    if kind == "sigmoid":
        e = np.exp(-np.abs(l))
        s, c = np.where(l < 0, e, 1.0) / (1.0 + e), np.where(l < 0, 1.0, e) / (1.0 + e)
    else:
        e = np.exp(l - l.max(1, keepdims=True))
        s, c = e / e.sum(1, keepdims=True), None
    return np.where(off, 0.0, s), c, off


def reference(g, l, idx, kind, normalize, scale):
    """(gradient, f G: what its float64 roundings are relative to)."""
    T, E = l.shape
    s, c, off = scores_of(l, kind)
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        sel = [(i, e) for i, e in enumerate(idx[t]) if 0 <= e < E and not off[t, e]]
        if not sel:
            continue
        gi, ei = np.array([g[t, i] for i, _ in sel]), np.array([e for _, e in sel])
        u = s[t, ei]
        if normalize:
            w, d, f = u / u.sum(), np.zeros(E), s[t] / u.sum()
            for i, e in enumerate(ei):
                d[e] += (w * (gi[i] - gi)).sum()
            f = np.where(np.isin(np.arange(E), ei), f, 0.0)
        else:
            d, f = np.zeros(E), s[t]
            np.add.at(d, ei, gi)
            if kind == "softmax":
                for e in range(E):
                    rest = s[t].sum() - s[t, e] if s[t, e] < 0.5 else np.delete(s[t], e).sum()
                    d[e] = d[e] * rest - (u * gi)[ei != e].sum()
        if kind == "sigmoid":
            f = f * c[t]
        cnt = np.bincount(ei, minlength=E) + (kind == "softmax" and not normalize)
        out[t] = np.where(off[t], 0.0, scale * f * d)
        mag[t] = f * np.abs(gi).max() * abs(scale) * cnt
    return out, mag


def check(torch, l, idx, kind, normalize, scale, index_type="int32", seed=9):
    l = np.asarray(l, np.float32)
    T, k = idx.shape
    U.say(f"[route scored grad] {l.shape} k={k} {kind} normalize={normalize}")
    g = np.random.default_rng(seed).standard_normal((T, k)).astype(np.float32)
    got = qm.route_scored_backward(torch.from_numpy(g).cuda(), torch.from_numpy(l).cuda(),
                                   torch.from_numpy(np.ascontiguousarray(idx.astype(index_type))).cuda(),
                                   {"scores": kind, "normalize_routing_weights": normalize, "scale": scale})
    ref, mag = reference(g.astype(np.float64), l.astype(np.float64), idx, kind, normalize, scale)
    if normalize:  # a row of one slot: nothing at all
        off = scores_of(l.astype(np.float64), kind)[2]
        one = [sum(0 <= e < l.shape[1] and not off[t, e] for e in idx[t]) == 1 for t in range(T)]
        assert not got.cpu().numpy()[one].any()
    U.check(U.back(got), ref, 2.0 ** -24 * (1 + 2.0 ** -20) * np.abs(ref) + (k + 16) * 2.0 ** -44 * mag + 2.0 ** -149, "grad_logits")


def largest(l, k):
    return np.argsort(-np.where(np.isnan(l), -np.inf, l), axis=1, kind="stable")[:, :k]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [1.0, 2.5, -0.3])
def test_a_single_slot_renormalised_has_no_gradient(torch, kind, scale):
    r = np.random.default_rng(1)
    l = r.standard_normal((4096, 33)) * 2
    idx = r.integers(0, 33, (4096, 1))
    check(torch, l, idx, kind, 1, scale)
    # the others masked or outside
    l[:, 7] = -np.inf
    l[:, 8] = np.nan
    idx = np.concatenate([np.full((4096, 1), 7), np.full((4096, 1), -1), r.integers(9, 33, (4096, 1)), np.full((4096, 2), 8)], 1)
    check(torch, l, idx, kind, 1, scale, "int64")
    # one expert in every slot
    check(torch, l, np.repeat(r.integers(9, 33, (4096, 1)), 5, 1), kind, 1, scale)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("normalize", [0, 1])
@pytest.mark.parametrize("T,E,k", [(2048, 64, 2), (2048, 128, 8), (512, 256, 6), (67, 300, 10), (40, 1024, 70), (130, 7, 7),
                                   (16, 65, 1), (1, 1, 1)])
def test_a_slot_that_dominates(torch, kind, normalize, T, E, k):
    # logits of spread 8: the first slot holds nearly all of the sum (softmax), or all slots differ by orders (sigmoid)
    r = np.random.default_rng(T + E + k)
    l = r.standard_normal((T, E)).astype(np.float32) * 8
    check(torch, l, largest(l, k), kind, normalize, 2.5, "int64" if E % 2 else "int32")
    if kind == "sigmoid":
        l = l - 30
        check(torch, l, largest(l, k), kind, normalize, 1.0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("normalize", [0, 1])
@pytest.mark.parametrize("E,k", [(6, 3), (70, 5), (200, 70), (1000, 300), (1024, 1024)])
def test_any_indices(torch, kind, normalize, E, k):
    # repeated, masked and outside ones
    r = np.random.default_rng(E + k)
    l = r.standard_normal((37, E)) * 6
    l[r.random(l.shape) < 0.1] = -np.inf
    l[5, 1:] = -np.inf
    l[6, 0] = np.nan
    idx = r.integers(-2, E + 2, (37, k))
    idx[1] = 4
    idx[2] = -1
    idx[3] = E
    idx[6, 0] = 0
    check(torch, l, idx, kind, normalize, 1.5, "int64" if E == 70 else "int32")


@pytest.mark.parametrize("kind", KINDS)
def test_scores_that_vanish_beside_others(torch, kind):
    # selected by a bias, their sum next to float32's smallest numbers: each slot's share is an ordinary number
    l = np.full((64, 16), 0.0, np.float32)
    l[:, :3] = -np.random.default_rng(3).uniform(70, 85, (64, 3))
    if kind == "softmax":
        l[:, 3:] = 0.0
    check(torch, l, np.tile(np.arange(3), (64, 1)), kind, 1, 2.0)
