"""Pins of the oracle of a routed layer's steps (CPU): against the whole
operator's oracle, and every gradient against central differences."""
import numpy as np
import pytest

import oracle
from oracle import steps_oracle as S

RNG = lambda s: np.random.default_rng(s)  # noqa: E731
H = 1e-6  # step of the central differences: truncation ~ H^2, rounding ~ 1e-16 / H = 1e-10


def _diff(f, a, g):
    """Central differences of <f(a), g> in every element of a."""
    out = np.zeros(a.shape)
    it = np.nditer(a, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        p, m = a.copy(), a.copy()
        p[i] += H
        m[i] -= H
        out[i] = np.sum((f(p) - f(m)) * g) / (2 * H)
    return out


@pytest.mark.parametrize("routing,normalize", [("qmoe", 0), ("moe", 0), ("moe", 1)])
def test_route_against_the_operator_and_differences(routing, normalize):
    r = RNG(1)
    logits = r.standard_normal((6, 9)).astype(np.float32).astype(np.float64)
    idx, w = S.route(logits, 3, routing, normalize)
    sel, ref = oracle.route(logits, 3, routing, normalize)
    np.testing.assert_array_equal(idx, sel)
    np.testing.assert_allclose(w, ref, rtol=1e-12)
    g = r.standard_normal(w.shape)
    grad = S.route_grad(g, logits, idx, routing, normalize)
    np.testing.assert_allclose(grad, _diff(lambda l: S.route(l, 3, routing, normalize)[1], logits, g), atol=1e-8)


def test_route_masked():
    ninf = -np.inf
    logits = np.array([[1.0, ninf, 2.0], [ninf, ninf, ninf], [ninf, np.nan, 0.5]])
    idx, w = S.route(logits, 2)
    np.testing.assert_array_equal(idx, [[2, 0], [-1, -1], [2, -1]])
    np.testing.assert_allclose(w[0].sum(), 1.0)
    np.testing.assert_array_equal(w[1:], [[0, 0], [1, 0]])


def test_dispatch_and_combine_are_each_others_transposes():
    r = RNG(2)
    T, k, E, Hd = 7, 3, 4, 5
    idx = r.integers(-1, E + 1, (T, k)).astype(np.int32)
    x = r.standard_normal((T, Hd))
    rows, off, perm, inv = S.dispatch(x, idx, E)
    assert sorted(perm) == list(range(T * k)) and off[-1] == np.sum((idx >= 0) & (idx < E))
    for e in range(E):
        s = perm[off[e]:off[e + 1]]
        assert np.all(idx.reshape(-1)[s] == e) and np.all(np.diff(s) > 0)
    # <dispatch(x), y> = <x, combine(y)>
    y = r.standard_normal(rows.shape)
    np.testing.assert_allclose(np.sum(rows * y), np.sum(x * S.combine(y, inv)))
    w = r.standard_normal((T, k))
    g = r.standard_normal((T, Hd))
    gr, gw = S.combine_grad(g, y, inv, w)
    np.testing.assert_allclose(gr, _diff(lambda a: S.combine(a, inv, w), y, g), atol=1e-8)
    np.testing.assert_allclose(gw, _diff(lambda a: S.combine(y, inv, a), w, g), atol=1e-8)


ATTRS = [("identity", {}), ("relu", {}), ("gelu", {}), ("silu", {}), ("swiglu", {}),
         ("swiglu", dict(alpha=1.7, beta=0.5, limit=0.8))]


@pytest.mark.parametrize("kind,a", ATTRS)
@pytest.mark.parametrize("grouped", [False, True])
def test_linear_gradients_against_differences(kind, a, grouped):
    r = RNG(3)
    M, K, N = 6, 4, 6
    x = r.standard_normal((M, K))
    w = r.standard_normal((3, N, K) if grouped else (N, K))
    b = r.standard_normal(w.shape[:-1])
    off = np.array([0, 2, 2, 5]) if grouped else None
    res = r.standard_normal((M, N // 2 if kind == "swiglu" else N))
    y, z = S.linear(x, w, b, res, off, kind, **a)
    g = r.standard_normal(y.shape)
    dx, dw, db, _ = S.linear_grad(g, x, w, z, off, kind, **a)
    f = lambda **kw: S.linear(kw.get("x", x), kw.get("w", w), kw.get("b", b), res, off, kind, **a)[0]  # noqa: E731
    np.testing.assert_allclose(dx, _diff(lambda v: f(x=v), x, g), atol=1e-7)
    np.testing.assert_allclose(dw, _diff(lambda v: f(w=v), w, g), atol=1e-7)
    np.testing.assert_allclose(db, _diff(lambda v: f(b=v), b, g), atol=1e-7)


def test_a_routed_layer_in_steps_is_the_float_moe():
    r = RNG(4)
    T, Hd, E, I, k = 9, 6, 4, 5, 2
    x, logits = r.standard_normal((T, Hd)), r.standard_normal((T, E))
    w1, b1 = r.standard_normal((E, 2 * I, Hd)), r.standard_normal((E, 2 * I))
    w2, b2 = r.standard_normal((E, Hd, I)), r.standard_normal((E, Hd))
    idx, w = S.route(logits, k, "moe", 0)
    rows, off, _, inv = S.dispatch(x, idx, E)
    h, _ = S.linear(rows, w1, b1, None, off, "swiglu")
    y, _ = S.linear(h, w2, b2, None, off)
    out = S.combine(y, inv, w)
    attrs = dict(k=k, activation_type="swiglu", swiglu_fusion=1)
    ref = oracle.moe(x, logits, w1, w2, fc1_b=b1, fc2_b=b2, attrs=attrs)
    np.testing.assert_allclose(out, ref, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("wrong", ["unstable", "no_mean", "gate_up_swapped"])
def test_planted_mistakes_fail(wrong, monkeypatch):
    r = RNG(5)
    if wrong == "unstable":
        idx = r.integers(0, 3, (8, 2)).astype(np.int32)
        _, perm, _ = S.sort_slots(idx, 3)
        bad = np.concatenate([np.flatnonzero(idx.reshape(-1) == e)[::-1] for e in range(3)])
        assert not np.array_equal(bad, perm)
    elif wrong == "no_mean":
        logits, g = r.standard_normal((4, 5)), r.standard_normal((4, 2))
        idx, w = S.route(logits, 2)
        bad = np.zeros((4, 5))
        np.put_along_axis(bad, idx.astype(np.int64), w * g, 1)
        assert np.abs(bad - S.route_grad(g, logits, idx)).max() > 1e-2
    else:
        z, dy = r.standard_normal((4, 6)), r.standard_normal((4, 3))
        sw = z.reshape(4, 3, 2)[:, :, ::-1].reshape(4, 6)
        assert np.abs(S.act(sw, "swiglu") - S.act(z, "swiglu")).max() > 1e-2
        assert np.abs(S.act_grad(dy, sw, "swiglu") - S.act_grad(dy, z, "swiglu")).max() > 1e-2
