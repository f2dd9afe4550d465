"""Norms whose result is an ordinary number though the products of its factors, taken in some order, are none: what the
weight times the row passes in float32's range, the weight times the normalised row (at most sqrt(H) in magnitude) does
not.  Bounds as in test_gpu_norm.py."""
import numpy as np
import pytest

import quantized_mixture_experts_router_amd as qm
from oracle import front_oracle as F

import front_util as V
import steps_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.skip("no GPU")
    return _t


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("H", [72, 1027, 33000])
@pytest.mark.parametrize("rows,weight,eps", [(1e15, 1e30, 1e-6), (1e-25, 1e-25, 1e-30), (1e15, 1e-30, 1e-6), (1e-18, 1e37, 1.0)])
def test_weight_times_row_beyond_float32(torch, dt, H, rows, weight, eps):
    U.say(f"[norm range {dt}] H={H} {rows} {weight} {eps}")
    r = np.random.default_rng(H)
    x, fx = U.typed(torch, r.standard_normal((3, H)) * rows, dt)
    w, fw = U.typed(torch, r.standard_normal(H) * weight, dt)
    y, _, codes, scales = qm.rms_norm(x, w, None, eps, "int8", 32)
    ref = F.rms_norm(fx, fw, eps)
    e = (H + 10) * 2.0 ** -24 * np.abs(ref)
    U.check(U.back(y), ref, U.rounded(dt, ref, e), "output")
    # (no scale is below 2^-126: what lies under half of that is 0)
    V.check_eight(torch, codes, scales, 32, ref, e + 2.0 ** -149, "8 bits")
