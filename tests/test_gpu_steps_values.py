"""Values at which the activations of the linear layers and their gradients
lose digits: far negative arguments of GELU."""
import math

import numpy as np
import pytest

import quantized_mixture_experts_router_amd as qm
from oracle import steps_oracle as S

import steps_util as U

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.skip("no GPU")
    return _t


def _column(torch, dt, z):
    """z as the pre-activation of a layer with one input and one column (products with 1 are exact)."""
    x, f = U.typed(torch, z.reshape(-1, 1), dt)
    return x, torch.ones(1, 1, dtype=x.dtype, device="cuda"), f


@pytest.mark.parametrize("dt", TYPES)
def test_gelu_far_below_zero(torch, dt):
    # gelu = z erfc(-z / sqrt 2) / 2 in float32.  The argument a = -z / sqrt 2 is two roundings off (the constant and the
    # product, 2^-24 relative each), and |a erfc'(a) / erfc(a)| <= 2 a^2 + 1 = z^2 + 1; erfc itself and the two products
    # around it: 32 steps.  The gradient adds z phi(z), whose exponent's rounding is at most z^2 2^-24 of it, to the same.
    z = np.concatenate([-np.linspace(3, 9, 4001), np.linspace(-3, 9, 2001)])
    x, w, f = _column(torch, dt, z)
    y = qm.linear(x, w, attrs={"activation_type": "gelu"})
    rel = 2.0 ** -24 * (2 * (f ** 2 + 1) + 32)
    ref = S.act(f, "gelu")
    U.check(U.back(y), ref, U.rounded(dt, ref, rel * np.abs(ref)), "gelu")
    one = torch.ones_like(x)
    _, _, gb = qm.linear_backward(one[:1], x[:1], w, x[:1], None, {"activation_type": "gelu"}, bias=True)
    gx, _, _ = qm.linear_backward(one, x, w, x, None, {"activation_type": "gelu"}, bias=True)
    gref = S.act_grad(np.ones_like(f), f, "gelu")
    mag = np.abs(S._phi(f)) + np.abs(f) * np.exp(-f * f / 2) / math.sqrt(2 * math.pi)
    e = rel * mag
    # (the gradient is rounded to the type as the operand of the product with 1, then the result: the same value)
    U.check(U.back(gx), gref, U.rounded(dt, gref, e), "gelu's gradient")
    U.check(U.back(gb), gref[0], U.rounded(dt, gref[0], e[0]), "bias gradient")
