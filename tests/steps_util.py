"""Helpers of the tests of a routed layer's steps: typed inputs with their
exact float64 values, and error bounds derived from the arithmetic.

Per element, with u the half step of the output type (float32 2^-24, float16
2^-11, bfloat16 2^-8: a rounding to nearest is off by at most u relative, or
by half a subnormal step), and A = sum_r |a_r b_r| the sum of magnitudes:
  - a float32 sum of n exact or float32-rounded products in any order is
    within e32 = 2 (n + 1) 2^-24 A of the exact one (n + 1 roundings of
    partial sums at most A, and their products' own, with a factor of two);
  - an activation maps an error e of its argument to at most its Lipschitz
    constant times e, plus the float32 evaluation of its formula.
"""
import numpy as np

HALF = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float32": 2.0 ** -149, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -133}  # half a subnormal step (f32, bf16: no less)
EV = 32 * 2.0 ** -24  # float32 evaluation of an activation: a dozen operations of at most 2 ulp each


def say(*a):
    print(*a, flush=True)


def typed(torch, a, dt, dev="cuda"):
    """(tensor of type dt, its exact float64 values)."""
    if a is None:
        return None, None
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float64)).to(getattr(torch, dt))
    return t.to(dev), t.to(torch.float64).numpy()


def back(t):
    return t.double().cpu().numpy()


def sum_bound(n, A):
    return 2.0 * (n + 1) * 2.0 ** -24 * A


def rounded(dt, ref, e):
    """Bound of a result within e of ref before its one rounding to dt."""
    return HALF[dt] * (np.abs(ref) + e) + TINY[dt] + e


def act_bound(z, ez, y, kind, alpha=1.0, beta=0.0, limit=None):
    """Error of act at arguments within ez of z, evaluated in float32."""
    if kind in ("identity", "relu"):
        return ez
    if kind in ("gelu", "silu"):
        # derivatives at most 1.13 and 1.1; the formulas' factors are at most |z|
        return 1.13 * ez + EV * np.abs(z)
    g, u = z[:, 0::2], z[:, 1::2]
    eg, eu = ez[:, 0::2], ez[:, 1::2]
    if limit is not None:
        g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
    # d/dg g sigma(alpha g) is at most 1.1, sigma at most 1
    return 1.1 * (np.abs(u + beta) + eu) * eg + (np.abs(g) + eg) * eu + EV * np.abs(g) * (np.abs(u) + abs(beta))


def grad_eval_bound(dy, z, kind, alpha=1.0, beta=0.0, limit=None):
    """Float32 evaluation error of act's gradient at exact arguments [M, N]."""
    if kind in ("identity", "relu"):
        return np.zeros(dy.shape if z is None else z.shape)
    if kind in ("gelu", "silu"):
        return EV * np.abs(dy) * (2.0 + np.abs(z))
    g, u = z[:, 0::2], z[:, 1::2]
    if limit is not None:
        g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
    e = np.zeros(z.shape)
    e[:, 0::2] = EV * np.abs(dy) * (np.abs(u) + abs(beta)) * (2.0 + np.abs(alpha * g))
    e[:, 1::2] = EV * np.abs(dy) * np.abs(g)
    return e


def check(got, ref, bound, label):
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    assert not np.isnan(got).any(), f"{label}: NaN (an element nothing wrote?)"
    err = np.abs(got - ref)
    worst = float((err / np.maximum(bound, 1e-300)).max()) if err.size else 0.0
    say(f"  {label}: max err / bound = {worst:.3g}")
    assert np.all(err <= bound), f"{label}: {worst} of the bound"
