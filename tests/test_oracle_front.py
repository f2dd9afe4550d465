"""Pins of the oracle of the norm, routing from scores and rows in 8 bits:
gradients against differences, formats against torch's type, corner cases by
hand, and mistakes planted in the oracle that make a pin fail."""
import math

import numpy as np
import pytest

from oracle import front_oracle as F


def RNG(s):
    return np.random.default_rng(s)


# ------------------------------------------------------------------ 8 bits
def test_e4m3_is_torchs_type():
    torch = pytest.importorskip("torch")
    codes = torch.arange(0x7f, dtype=torch.uint8)
    np.testing.assert_array_equal(codes.view(torch.float8_e4m3fn).float().numpy(), F.e4m3_values())
    q = np.concatenate([RNG(1).standard_normal(500) * 50, np.array(F.e4m3_values()) * 1.0, [464.0, -464.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    q = q.astype(np.float32)
    want = torch.from_numpy(q).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal([F.round_e4m3(float(v)) for v in q], want)


@pytest.mark.parametrize("fmt,top", [("int8", 127), ("e4m3", 448)])
def test_scale_is_the_least(fmt, top):
    for m in (1.0, 127.0, 127.49999, 127.5, 128.0, 463.9, 464.0, 464.1, 3e38, 1e-3, 1e-30, 1e-45):
        e = F.scale_exponent(m, fmt)
        q = round(m / 2.0 ** e) if fmt == "int8" else F.round_e4m3(m / 2.0 ** e)
        assert q <= top
        if e > -126:  # at half the scale the largest value has no code
            over = m / 2.0 ** (e - 1)
            assert (round(over) if fmt == "int8" else over) > (top if fmt == "int8" else 464.0)


def test_rows_in_8_bits_by_hand():
    v, s = F.eight(np.array([[1.0, -3.5, 0.5, 200.0], [0.0, 0.0, 0.0, 0.0], [1.0, np.inf, 2.0, 3.0]]), "int8", 2)
    np.testing.assert_array_equal(s, [[2.0 ** -5, 2.0], [1.0, 1.0], [np.nan, 2.0 ** -5]])
    np.testing.assert_array_equal(v[0], [1.0, -3.5, 0.0, 200.0])  # 0.25 rounds to 0
    assert not v[1].any() and np.isnan(v[2, :2]).all()
    np.testing.assert_array_equal(v[2, 2:], [2.0, 3.0])
    # an odd half rounds to the even code
    v, s = F.eight(np.array([[127.0, 2.5, 3.5, -2.5]]), "int8", 16)
    np.testing.assert_array_equal(v, [[127.0, 2.0, 4.0, -2.0]])


def test_errors_of_8_bits_are_half_a_step():
    x = RNG(2).standard_normal((20, 70)) * np.exp(RNG(3).standard_normal(70))
    for fmt in ("int8", "e4m3"):
        v, s = F.eight(x, fmt, 32)
        step = np.repeat(s, 32, axis=1)[:, :70]
        half = step / 2 if fmt == "int8" else np.maximum(np.abs(x) * 2.0 ** -4, step * 2.0 ** -10)
        assert (np.abs(v - x) <= half).all()


def test_codes_stand_for_their_values():
    c = np.array([[128, 255, 1, 0x80 | 0x08]], np.uint8)
    np.testing.assert_array_equal(F.values(c, np.array([[0.5]]), "int8", 16), [[0.0, 63.5, -63.5, 4.0]])
    c = np.array([[0, 0x38, 0xb8, 0x7e]], np.uint8)
    np.testing.assert_array_equal(F.values(c, np.array([[2.0]]), "e4m3", 16), [[0.0, 2.0, -2.0, 896.0]])


def test_slots_take_their_tokens_rows():
    rows = np.array([[1.0], [2.0], [3.0]])
    np.testing.assert_array_equal(F.slots(rows, [5, 0, 2, -1, 3, 6], 2), [[3.0], [1.0], [2.0], [0.0], [2.0], [0.0]])


# ------------------------------------------------------------------ norm
def test_norm_by_hand():
    y = F.rms_norm(np.array([[3.0, 4.0], [0.0, 0.0]]), np.array([1.0, 2.0]), 0.5)
    s = 1 / math.sqrt(12.5 + 0.5)
    np.testing.assert_allclose(y, [[3 * s, 8 * s], [0, 0]], rtol=1e-15)


def test_norm_gradients_against_differences():
    r = RNG(4)
    for H in (1, 5, 8):
        h, w, dy, ds = r.standard_normal((3, H)), r.standard_normal(H), r.standard_normal((3, H)), r.standard_normal((3, H))

        def loss(h, w):
            return float((F.rms_norm(h, w, 0.3) * dy).sum() + (ds * h).sum())
        dh, dw = F.rms_norm_grad(dy, h, w, ds, 0.3)
        d = 1e-5
        for at in np.ndindex(h.shape):
            e = np.zeros(h.shape)
            e[at] = d
            assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * d) - dh[at]) < 1e-8
        for c in range(H):
            e = np.zeros(H)
            e[c] = d
            assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * d) - dw[c]) < 1e-8


# ------------------------------------------------------------------ routing
def test_route_by_hand():
    l = np.array([[0.0, 1.0, 2.0, 3.0, 4.0, 5.0]])
    idx, w = F.route_scored(l, 2, "sigmoid")
    np.testing.assert_array_equal(idx, [[5, 4]])
    np.testing.assert_allclose(w, [[1 / (1 + math.exp(-5)), 1 / (1 + math.exp(-4))]], rtol=1e-7)
    # the bias selects but does not weigh
    idx, w = F.route_scored(l, 2, "sigmoid", bias=np.array([9.0, 0, 0, 0, 0, 0]), normalize=1, scale=3.0)
    np.testing.assert_array_equal(idx, [[0, 5]])
    s = [0.5, 1 / (1 + math.exp(-5))]
    np.testing.assert_allclose(w, [[3 * s[0] / sum(s), 3 * s[1] / sum(s)]], rtol=1e-7)
    # groups of two: by the largest the last, by the sum of two the middle one
    l = np.array([[0.0, 0.0, 2.0, 2.0, -9.0, 3.0]])
    assert F.route_scored(l, 1, "sigmoid", groups=3, kept=1, group_top=1)[0] == [[5]]
    assert F.route_scored(l, 1, "sigmoid", groups=3, kept=1, group_top=2)[0] == [[2]]


def test_route_masks():
    n = -np.inf
    l = np.array([[n, n, n, n], [1.0, n, np.nan, n], [n, 1.0, 2.0, np.inf]])
    for kind in ("softmax", "sigmoid"):
        idx, w = F.route_scored(l, 2, kind, normalize=1)
        # (beside an infinite logit the softmax leaves the others 0 each: the lower one)
        np.testing.assert_array_equal(idx, [[-1, -1], [0, -1], [3, 1 if kind == "softmax" else 2]])
        assert w[0].tolist() == [0, 0] and w[1].tolist() == [1, 0]
    idx, _ = F.route_scored(l, 2, "sigmoid", bias=np.array([0, 0, n, np.nan]))
    np.testing.assert_array_equal(idx, [[-1, -1], [0, -1], [1, -1]])
    # a group without experts ranks last, one with a single expert by it alone
    idx, _ = F.route_scored(np.array([[n, n, -3.0, n, -4.0, -4.0]]), 1, "softmax", groups=3, kept=1, group_top=2)
    np.testing.assert_array_equal(idx, [[2]])


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [0, 1])
def test_route_gradient_against_differences(kind, normalize):
    r = RNG(6)
    l = r.standard_normal((4, 6))
    l[1, 2] = -np.inf
    idx, _ = F.route_scored(l, 3, kind, normalize=normalize)
    idx[2, 1] = -1
    idx[3, 1] = idx[3, 0]
    g = r.standard_normal((4, 3))

    def loss(l):
        s, _ = F.scores(l, kind)
        total = 0.0
        for t in range(4):
            sel = [(i, e) for i, e in enumerate(idx[t]) if e >= 0]
            S = sum(s[t, e] for _, e in sel) if normalize else 1.0
            total += sum(g[t, i] * 2.5 * s[t, e] / S for i, e in sel)
        return total
    got = F.route_scored_grad(g, l, idx, kind, normalize, 2.5)
    for at in np.ndindex(l.shape):
        if not np.isfinite(l[at]):
            assert got[at] == 0
            continue
        e = np.zeros(l.shape)
        e[at] = 1e-5
        assert abs((loss(l + e) - loss(l - e)) / 2e-5 - got[at]) < 1e-6  # (scores rounded to float32)


# ------------------------------------------------------------------ planted mistakes
PINS = [lambda: test_scale_is_the_least("int8", 127), lambda: test_scale_is_the_least("e4m3", 448),
        test_rows_in_8_bits_by_hand, test_errors_of_8_bits_are_half_a_step, test_codes_stand_for_their_values,
        test_slots_take_their_tokens_rows, test_norm_by_hand, test_norm_gradients_against_differences,
        test_route_by_hand, test_route_masks,
        *[lambda k=k, n=n: test_route_gradient_against_differences(k, n) for k in ("softmax", "sigmoid") for n in (0, 1)]]


def pins_pass():
    try:
        for p in PINS:
            p()
    except Exception:  # an assertion, or an error that the mistake leads to
        return False
    return True


MISTAKES = {
    "scale one too large": ("scale_exponent", lambda f: lambda m, fmt: f(m, fmt) + 1),
    "scale of the largest code": ("scale_exponent", lambda f: lambda m, fmt: f(m * 1.0041, fmt)),
    "code 127 for zero": ("values", lambda f: lambda c, s, fmt, b: f(c, s, fmt, b) + (s[0, 0] if fmt == "int8" else 0)),
    "slot for token": ("slots", lambda f: lambda r, p, k: f(r, p, 1)),
    "mean without epsilon": ("rms_norm", lambda f: lambda h, w=None, eps=1e-6: f(h, w, 0.0)),
    "weight outside the mean": ("rms_norm_grad", lambda f: lambda dy, h, w=None, ds=None, eps=1e-6:
                                (f(dy, h, None, ds, eps)[0] * w, f(dy, h, w, ds, eps)[1])),
    "bias weighs": ("route_scored", lambda f: lambda l, k, kind="softmax", bias=None, **a:
                    f(l if bias is None else l + np.nan_to_num(bias), k, kind, None, **a)),
    "ties to the higher": ("route_scored", lambda f: lambda l, k, *a, **b: (l.shape[1] - 1 - f(l[:, ::-1], k, *a, **b)[0], 0)),
    "renormalised as if constant": ("route_scored_grad", lambda f: lambda g, l, i, kind="softmax", normalize=0, scale=1.0:
                                    f(g, l, i, kind, 0, scale)),
    "no scale": ("route_scored_grad", lambda f: lambda g, l, i, kind="softmax", normalize=0, scale=1.0:
                 f(g, l, i, kind, normalize, 1.0)),
}


def test_pins_pass_without_a_mistake():
    assert pins_pass()


@pytest.mark.parametrize("name", MISTAKES)
def test_planted_mistake_is_caught(monkeypatch, name):
    at, change = MISTAKES[name]
    monkeypatch.setattr(F, at, change(getattr(F, at)))
    assert not pins_pass()
