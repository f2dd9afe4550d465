"""Mistakes planted in the oracle of a routed layer's steps: each makes a pin
fail (the pins of test_oracle_steps, and the ones below)."""
import numpy as np
import pytest

from oracle import steps_oracle as S

import test_oracle_steps as P


def test_route_ties_go_to_the_lower_expert():
    idx, w = S.route(np.array([[1.0, 2.0, 2.0, 2.0], [3.0, 3.0, 0.0, 3.0]]), 2)
    np.testing.assert_array_equal(idx, [[1, 2], [0, 1]])
    np.testing.assert_allclose(w, 0.5)


def test_rows_behind_the_last_group_are_zero():
    r = P.RNG(7)
    x, w, b, res = r.standard_normal((6, 3)), r.standard_normal((2, 4, 3)), r.standard_normal((2, 4)), r.standard_normal((6, 4))
    off = np.array([0, 1, 4])
    y, z = S.linear(x, w, b, res, off, "relu")
    assert not y[4:].any() and not z[4:].any()
    np.testing.assert_allclose(y[1:4], np.maximum(x[1:4] @ w[1].T + b[1], 0) + res[1:4])
    dx, dw, db, _ = S.linear_grad(res, x, w, z, off, "identity")
    assert not dx[4:].any()
    np.testing.assert_allclose(db[1], res[1:4].sum(0))


def test_dropped_slots_lie_behind_the_last_expert_in_order():
    off, perm, inv = S.sort_slots(np.array([[2, -1], [0, 5], [2, 0]]), 3)
    np.testing.assert_array_equal(off, [0, 2, 2, 4])
    np.testing.assert_array_equal(perm, [2, 5, 0, 4, 1, 3])
    np.testing.assert_array_equal(inv, [[2, -5], [0, -6], [3, 1]])


def pins_pass():
    try:
        for routing, normalize in (("qmoe", 0), ("moe", 0), ("moe", 1)):
            P.test_route_against_the_operator_and_differences(routing, normalize)
        P.test_route_masked()
        P.test_dispatch_and_combine_are_each_others_transposes()
        for kind, a in P.ATTRS:
            for grouped in (False, True):
                P.test_linear_gradients_against_differences(kind, a, grouped)
        P.test_a_routed_layer_in_steps_is_the_float_moe()
        test_route_ties_go_to_the_lower_expert()
        test_rows_behind_the_last_group_are_zero()
        test_dropped_slots_lie_behind_the_last_expert_in_order()
    except Exception:  # an assertion, or an error that the mistake leads to
        return False
    return True


def _plant(monkeypatch, mistake):
    route, route_grad, sort_slots = S.route, S.route_grad, S.sort_slots
    combine, combine_grad, act, act_grad, preact = S.combine, S.combine_grad, S.act, S.act_grad, S.preact

    def put(name, f):
        monkeypatch.setattr(S, name, f)
    if mistake == "ties to the higher expert":
        def f(l, k, routing="qmoe", normalize=0):
            i, w = route(l[:, ::-1], k, routing, normalize)
            return np.where(i < 0, -1, l.shape[1] - 1 - i).astype(np.int32), w
        put("route", f)
    elif mistake == "weights over all experts":
        put("route", lambda l, k, routing="qmoe", normalize=0: route(l, k, "moe", 0))
    elif mistake == "gradient without the mean":
        def f(g, l, i, routing="qmoe", normalize=0):
            out = np.zeros(l.shape)
            np.put_along_axis(out, i.astype(np.int64), S.route(l, i.shape[1], routing, normalize)[1] * g, 1)
            return out
        put("route_grad", f)
    elif mistake == "gradient over the selection alone":
        put("route_grad", lambda g, l, i, routing="qmoe", normalize=0: route_grad(g, l, i, "qmoe", 0))
    elif mistake == "slots of an expert backwards":
        def f(i, experts):
            off, perm, _ = sort_slots(i, experts)
            perm = np.concatenate([perm[off[e]:off[e + 1]][::-1] for e in range(experts)] + [perm[off[-1]:]])
            inv = np.zeros(i.size, np.int32)
            for p, s in enumerate(perm):
                inv[s] = p if p < off[-1] else -1 - p
            return off, perm, inv.reshape(i.shape)
        put("sort_slots", f)
    elif mistake == "dropped slots backwards":
        def f(i, experts):
            off, perm, inv = sort_slots(i, experts)
            n, S_ = off[-1], i.size
            perm = np.concatenate([perm[:n], perm[n:][::-1]])
            return off, perm, np.where(inv < 0, -1 - (n + S_ - 1 - (-1 - inv)), inv).astype(np.int32)
        put("sort_slots", f)
    elif mistake == "combine without weights":
        put("combine", lambda rows, inverse, weights=None: combine(rows, inverse))
    elif mistake == "weight gradient of the next token":
        def f(g, rows, inverse, weights):
            return combine_grad(g, rows, inverse, weights)[0], combine_grad(np.roll(g, 1, 0), rows, inverse, weights)[1]
        put("combine_grad", f)
    elif mistake == "gate and linear branch swapped":
        def f(z, kind, **a):
            return act(z.reshape(len(z), -1, 2)[:, :, ::-1].reshape(z.shape) if kind == "swiglu" else z, kind, **a)
        put("act", f)
    elif mistake == "silu's gradient without its second term":
        put("act_grad", lambda dy, z, kind, **a: dy * S._sigma(z) if kind == "silu" else act_grad(dy, z, kind, **a))
    elif mistake == "gradient through the limit":
        def f(dy, z, kind, **a):
            return act_grad(dy, z, kind, **{n: v for n, v in a.items() if n != "limit"})
        put("act_grad", f)
    elif mistake == "relu's gradient everywhere":
        put("act_grad", lambda dy, z, kind, **a: dy.copy() if kind == "relu" else act_grad(dy, z, kind, **a))
    elif mistake == "every group with the first one's bias":
        put("preact", lambda x, w, b, offsets=None: preact(
            x, w, b if b is None or w.ndim == 2 else np.repeat(b[:1], len(w), 0), offsets))
    elif mistake == "residual behind the last group":
        put("live_rows", lambda M, w, offsets: M)


MISTAKES = ["ties to the higher expert", "weights over all experts", "gradient without the mean",
            "gradient over the selection alone", "slots of an expert backwards", "dropped slots backwards",
            "combine without weights", "weight gradient of the next token", "gate and linear branch swapped",
            "silu's gradient without its second term", "gradient through the limit", "relu's gradient everywhere",
            "every group with the first one's bias", "residual behind the last group"]


def test_pins_pass_without_a_mistake():
    assert pins_pass()


@pytest.mark.parametrize("mistake", MISTAKES)
def test_a_planted_mistake_fails_a_pin(monkeypatch, mistake):
    _plant(monkeypatch, mistake)
    assert not pins_pass()
