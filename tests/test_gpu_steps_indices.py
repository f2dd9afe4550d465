"""Router gradients over indices that no forward pass gives: an expert twice,
outside the experts, masked, in every routing mode."""
import numpy as np
import pytest

import quantized_mixture_experts_router_amd as qm
from oracle import steps_oracle as S

import steps_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.skip("no GPU")
    return _t


@pytest.mark.parametrize("index_type", ["int32", "int64"])
@pytest.mark.parametrize("routing,normalize", [("qmoe", 0), ("moe", 0), ("moe", 1)])
@pytest.mark.parametrize("E,k", [(6, 3), (70, 5), (200, 70)])
def test_route_backward_over_any_indices(torch, routing, normalize, E, k, index_type):
    # softmax over the selection: an expert taken twice counts twice in the sum as well as in the gradient
    r = np.random.default_rng(E + k)
    T = 37
    l = r.standard_normal((T, E)).astype(np.float32)
    l[r.random(l.shape) < 0.1] = -np.inf
    l[5] = -np.inf
    l[6, 0] = np.nan
    idx = r.integers(-2, E + 2, (T, k))
    idx[1] = 4
    idx[2] = -1
    idx[3] = E
    idx[6, 0] = 0
    g = r.standard_normal((T, k)).astype(np.float32)
    a = {"k": k, "routing": routing, "normalize_routing_weights": normalize}
    U.say(f"[route grad] E={E} k={k} {routing} {normalize} {index_type}")
    got = qm.route_backward(torch.from_numpy(g).cuda(), torch.from_numpy(l).cuda(),
                            torch.from_numpy(idx).to(getattr(torch, index_type)).cuda(), a)
    ref = S.route_grad(g.astype(np.float64), l.astype(np.float64), idx, routing, normalize)
    # every weight is within 2 2^-24 (spread + E + 16) of itself (exp of a rounded difference, a sum of at most E terms,
    # a division); the gradient is a sum of at most k products of them with g and g - mean
    spread = 8.0  # (logits within +-4)
    assert np.abs(l[np.isfinite(l)]).max() < 4.5
    rel = 2 * 2.0 ** -24 * (spread + max(E, k) + 16)
    bound = 4 * rel * 2 * np.abs(g).max() + k * 2.0 ** -24 * np.abs(g).max()
    U.check(U.back(got), ref, np.full(ref.shape, bound), "grad_logits")
