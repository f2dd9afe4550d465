"""GPU parity of routing from scores and its gradient with the float64 oracle:
indices exact, weights and gradients to bounds derived from the arithmetic."""
import numpy as np
import pytest

import quantized_mixture_experts_router_amd as qm
from oracle import front_oracle as F

import steps_util as U

pytestmark = pytest.mark.gpu

NINF = -np.inf
u = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.skip("no GPU")
    return _t


def check(torch, l, k, kind, bias=None, groups=1, kept=1, group_top=2, normalize=0, scale=1.0, index_type="int32", idx=None):
    l = np.asarray(l, np.float32)
    T, E = l.shape
    U.say(f"[route scored] {l.shape} k={k} {kind} groups={groups}/{kept}/{group_top} normalize={normalize}")
    a = {"k": k, "scores": kind, "groups": groups, "kept_groups": kept, "group_top": group_top,
         "normalize_routing_weights": normalize, "scale": scale}
    tl = torch.from_numpy(l).cuda()
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    got, w = qm.route_scored(tl, b, a)
    torch.cuda.synchronize()
    ri, rw = F.route_scored(l.astype(np.float64), k, kind, None if b is None else b.double().cpu().numpy(), groups, kept,
                            group_top, normalize, scale)
    np.testing.assert_array_equal(got.cpu().numpy(), ri)
    # the scores are float32's nearest; renormalised: a sum of k of them, a division; the scale
    U.check(U.back(w), rw, (2 * k + 8) * u * np.abs(rw) + 2.0 ** -126 * max(1.0, abs(scale)), "weights")
    g = np.random.default_rng(9).standard_normal((T, k)).astype(np.float32)
    i = ri if idx is None else idx
    gl = qm.route_scored_backward(torch.from_numpy(g).cuda(), tl, torch.from_numpy(i.astype(index_type)).cuda(), a)
    ref = F.route_scored_grad(g.astype(np.float64), l, i, kind, normalize, scale)
    # a score is within rel of itself: an exponential of a (rounded) argument, for the softmax a sum of E terms, a division
    s, off = F.scores(l.astype(np.float64), kind)
    fin = np.where(np.isfinite(l), l, 0.0)
    spread = (fin.max(1) - fin.min(1)).clip(max=200.0) if kind == "softmax" else np.zeros(T)
    rel = (2 * u * (spread + (E if kind == "softmax" else 0) + 16))[:, None]
    rel = rel + 2.0 ** -148 / np.maximum(s, 2.0 ** -148)  # a step of float32's subnormal numbers
    G = np.abs(g).max(1, keepdims=True) * abs(scale)
    cnt = np.zeros((T, E))
    S, worst = np.zeros((T, 1)), np.zeros((T, 1))
    for t in range(T):
        for e in i[t]:
            if 0 <= e < E and not off[t, e]:
                cnt[t, e] += 1
                S[t] += np.float32(s[t, e])
                worst[t] = max(worst[t, 0], rel[t, e])
    rel = rel + worst
    f = np.where(S > 0, s / np.where(S > 0, S, 1), 0) if normalize else s
    # gradient = f (sum of the expert's slots' (g - shift) - mean): shift and mean sums of k products of scores, 2 G and k G at most
    bound = f * 2 * G * (cnt + (k if kind == "softmax" and not normalize else 0)) * (8 * rel + 16 * (k + 4) * u)
    if kind == "softmax" and not normalize:
        bound += s * G * np.minimum(k, S) * (8 * rel + 16 * (k + 4) * u)
    # the definition's own float64 rounding: where the renormalised softmax's sum of k terms of at most 2 G f cancels to 0,
    # k roundings of 2^-53 of a partial sum and as many of its terms are left in every expert's s times it
    bound += f * G * 4 * (k + 4) * 2.0 ** -52
    U.check(U.back(gl), ref, bound + 2.0 ** -120, "grad_logits")


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [0, 1])
@pytest.mark.parametrize("T,E,k,groups,kept", [(1, 1, 1, 1, 1), (16, 8, 2, 1, 1), (5, 7, 7, 7, 7), (67, 64, 6, 8, 3), (130, 65, 8, 5, 2),
                                               (33, 128, 8, 8, 4), (9, 300, 10, 3, 1), (3, 1024, 70, 64, 9), (2, 129, 129, 1, 1),
                                               (21, 256, 8, 8, 4), (6, 512, 4, 16, 16), (4, 96, 1, 48, 1), (7, 60, 20, 60, 25)])
def test_route(torch, kind, normalize, T, E, k, groups, kept):
    r = np.random.default_rng(T * E + k)
    top = 1 + (T + k) % 2
    it = "int64" if E % 2 else "int32"
    check(torch, r.standard_normal((T, E)) * 2, k, kind, None, groups, kept, top, normalize, 1.0, it)
    b = r.standard_normal(E) * 0.1
    check(torch, r.standard_normal((T, E)) * 2, k, kind, b, groups, kept, 3 - top, normalize, 2.5, it)
    # few distinct values: ties everywhere, among experts and among groups
    check(torch, r.integers(-1, 2, (T, E)) * 1.0, k, kind, r.integers(0, 2, E) * 0.25, groups, kept, top, normalize, 1.0, it)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [0, 1])
@pytest.mark.parametrize("groups,kept,top", [(1, 1, 2), (7, 3, 2), (7, 3, 1), (14, 2, 2)])
def test_masks(torch, kind, normalize, groups, kept, top):
    r = np.random.default_rng(3)
    l = r.standard_normal((40, 70))
    l[r.random(l.shape) < 0.8] = NINF
    l[3] = NINF
    l[4, 1:] = NINF
    l[5] = np.nan
    l[6, ::2] = np.nan
    l[7] = np.finfo(np.float32).min  # the type's lowest value masks nothing
    l[8, :60] = np.finfo(np.float32).min
    l[9] = 1e30
    l[10, 5] = np.inf
    l[11, [3, 60]] = np.inf
    l[12] = np.inf
    check(torch, l, 5, kind, None, groups, kept, top, normalize)
    b = r.standard_normal(70) * 0.2
    b[[0, 30, 31]] = NINF
    b[7] = np.nan
    b[12] = np.inf
    check(torch, l, 5, kind, b, groups, kept, top, normalize, 1.5)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_scores_that_differ_in_the_last_bits(torch, kind):
    # the neighbours of one score, ranked: a float32 exponential would swap some of them
    r = np.random.default_rng(8)
    l = np.nextafter(np.float32(0.7), np.float32(2), dtype=np.float32) + r.integers(0, 40, (200, 128)).astype(np.float32) * 2.0 ** -24
    check(torch, l, 16, kind)
    check(torch, l, 16, kind, r.integers(0, 3, 128) * 2.0 ** -24, 8, 4)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [0, 1])
def test_scores_near_zero(torch, kind, normalize):
    # selected by the bias, with scores that vanish beside the others'
    l = np.array([[-100.0, 0.0, -101.0, -150.0], [-90.0, -88.0, -200.0, -300.0], [-800.0, -900.0, -1e30, -2e38], [88.0, 90.0, 200.0, 3e38]])
    check(torch, l, 2, kind, np.array([9.0, 0.0, 8.0, 0.0]), normalize=normalize, scale=2.0)


@pytest.mark.parametrize("index_type", ["int32", "int64"])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [0, 1])
@pytest.mark.parametrize("E,k", [(6, 3), (70, 5), (200, 70)])
def test_gradient_over_any_indices(torch, kind, normalize, E, k, index_type):
    r = np.random.default_rng(E + k)
    T = 37
    l = r.standard_normal((T, E))
    l[r.random(l.shape) < 0.1] = NINF
    l[5] = NINF
    l[6, 0] = np.nan
    idx = r.integers(-2, E + 2, (T, k))
    idx[1] = 4
    idx[2] = -1
    idx[3] = E
    idx[6, 0] = 0
    check(torch, l, k, kind, normalize=normalize, scale=1.5, index_type=index_type, idx=idx)


def test_indices_beyond_32_bits_are_outside(torch):
    l = torch.zeros(2, 4, device="cuda")
    idx = torch.tensor([[1 << 32], [(1 << 32) + 1]], device="cuda")
    assert not qm.route_scored_backward(torch.ones(2, 1, device="cuda"), l, idx, {"scores": "sigmoid"}).any()


def test_without_bias_and_groups_it_is_route(torch):
    # the softmax over all experts of qmoe_route (whose weights are float32 all through)
    r = np.random.default_rng(5)
    l = torch.from_numpy(r.standard_normal((300, 96)).astype(np.float32)).cuda()
    for n in (0, 1):
        i, w = qm.route_scored(l, None, {"k": 6, "normalize_routing_weights": n})
        j, v = qm.route(l, {"k": 6, "routing": "moe", "normalize_routing_weights": n})
        assert torch.equal(i, j)
        assert float(((w - v) / v).abs().max()) <= 4 * u * (8 + 96 + 16)


def test_of_2_to_the_26_tokens(torch):
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GiB of GPU memory")
    T = (1 << 26) + 5
    U.say(f"[route scored] T={T}")
    l = torch.randn(T, 2, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    a = {"k": 1, "scores": "sigmoid"}
    idx, w = qm.route_scored(l, None, a)
    s = (1 / (1 + torch.exp(-l.double()))).float()
    second = s[:, 1] > s[:, 0]
    assert torch.equal(idx[:, 0] == 1, second)
    assert float((w[:, 0] - torch.maximum(s[:, 0], s[:, 1])).abs().max()) <= u
    gl = qm.route_scored_backward(torch.full((T, 1), 2.0, device="cuda"), l, idx, a)
    ref = torch.where(torch.stack([~second, second], 1), 2 * s * (1 - s), 0.0)
    assert float((gl - ref).abs().max()) <= 64 * u
