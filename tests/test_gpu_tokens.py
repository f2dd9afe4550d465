"""GPU parity of routing weights, token dispatch and combine, each with its
gradient, with the float64 oracle (bounds of steps_util; indices and sorted
orders exact)."""
import numpy as np
import pytest

import quantized_mixture_experts_router_amd as qm
from oracle import steps_oracle as S

import steps_util as U

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]
ROUTING = [("qmoe", 0), ("moe", 0), ("moe", 1)]
NINF = -np.inf


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.skip("no GPU")
    return _t


def _attrs(k, routing, normalize):
    return {"k": k, "routing": routing, "normalize_routing_weights": normalize}


def _check_route(torch, logits, k, routing, normalize, index_type="int32"):
    a = _attrs(k, routing, normalize)
    l = torch.from_numpy(logits.astype(np.float32)).cuda()
    f = logits.astype(np.float32).astype(np.float64)
    U.say(f"[route] {logits.shape} k={k} {routing} {normalize}")
    idx, w = qm.route(l, a)
    torch.cuda.synchronize()
    ri, rw = S.route(f, k, routing, normalize)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    # exp of a difference (rounded, relative 2^-24 of the difference's magnitude times it), a sum of at most E terms
    # and a division
    spread = np.max(np.where(np.isfinite(f), f, 0), 1) - np.min(np.where(np.isfinite(f), f, 0), 1)
    rel = (2.0 ** -24 * (spread + f.shape[1] + 16))[:, None] * 2
    U.check(U.back(w), rw, rel * rw + 2.0 ** -126, "weights")
    g = np.random.default_rng(9).standard_normal(rw.shape).astype(np.float32)
    gl = qm.route_backward(torch.from_numpy(g).cuda(), l, idx.to(getattr(torch, index_type)), a)
    ref = S.route_grad(g.astype(np.float64), f, ri, routing, normalize)
    mag = np.abs(rw * g).sum(1, keepdims=True)
    # w (g - mean): w as above, mean a sum of at most k products
    U.check(U.back(gl), ref, 4 * rel * (mag + np.abs(g).max(1, keepdims=True) * 1.0) + 2.0 ** -126, "grad_logits")


@pytest.mark.parametrize("routing,normalize", ROUTING)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (16, 8, 2), (5, 7, 7), (67, 64, 6), (130, 65, 8), (33, 128, 8),
                                   (9, 300, 10), (3, 1024, 70), (2, 129, 129)])
def test_route(torch, routing, normalize, T, E, k):
    r = np.random.default_rng(T * E)
    _check_route(torch, r.standard_normal((T, E)) * 2, k, routing, normalize, "int64" if E % 2 else "int32")
    # few distinct values: ties everywhere
    _check_route(torch, r.integers(-1, 2, (T, E)) * 1.0, k, routing, normalize)


@pytest.mark.parametrize("routing,normalize", ROUTING)
def test_route_masked_experts(torch, routing, normalize):
    r = np.random.default_rng(3)
    l = r.standard_normal((40, 70))
    l[r.random(l.shape) < 0.9] = NINF
    l[3] = NINF
    l[4, 1:] = NINF
    l[5] = np.nan
    l[6, ::2] = np.nan
    l[7] = np.finfo(np.float32).min  # the type's lowest value masks nothing
    l[8, :60] = np.finfo(np.float32).min
    l[9] = 1e30
    _check_route(torch, l, 5, routing, normalize)


def test_route_is_the_operators(torch):
    # the selection and weights of the whole operator's router
    from quantized_mixture_experts_router_amd import workloads as W
    for routing, normalize in ROUTING:
        wl, a = W.random_case(np.random.default_rng(1), tokens_shape=(50,), hidden=32, experts=16, inter=32, k=3,
                              bits=8, block_size=0, activation="relu")
        attrs = dict(wl.attrs(), routing=routing, normalize_routing_weights=normalize)
        d = {n: torch.from_numpy(v).cuda() for n, v in a.items()}
        dbg = {"topk_idx": torch.empty(150, dtype=torch.int32, device="cuda"),
               "topk_w": torch.empty(150, dtype=torch.float32, device="cuda")}
        qm.forward(*d.values(), attrs, debug=dbg)
        idx, w = qm.route(d["router_probs"], attrs)
        torch.cuda.synchronize()
        assert torch.equal(idx.view(-1), dbg["topk_idx"])
        assert float((w.view(-1) - dbg["topk_w"]).abs().max()) <= 1e-6


def test_route_backward_takes_any_indices(torch):
    # the same expert twice adds twice; outside [0, E) adds nothing
    l = np.random.default_rng(1).standard_normal((4, 6)).astype(np.float32)
    idx = np.array([[1, 1, 2], [5, -1, 9], [0, 3, 3], [-1, -1, -1]], np.int64)
    g = np.random.default_rng(2).standard_normal((4, 3)).astype(np.float32)
    for routing in ("moe",):
        got = qm.route_backward(torch.from_numpy(g).cuda(), torch.from_numpy(l).cuda(), torch.from_numpy(idx).cuda(),
                                _attrs(3, routing, 0))
        ref = S.route_grad(g.astype(np.float64), l.astype(np.float64), idx, routing, 0)
        U.check(U.back(got), ref, np.full(ref.shape, 64 * 2.0 ** -24), "grad_logits")


# ------------------------------------------------------------------ dispatch and combine
def _indices(r, T, k, E, kind):
    if kind == "one":  # every slot to one expert
        return np.full((T, k), E // 2, np.int64)
    if kind == "none":
        return np.full((T, k), -1, np.int64)
    if kind == "wild":  # dropped slots of every kind
        i = r.integers(-3, E + 3, (T, k))
        i[r.random(i.shape) < 0.05] = 2 ** 31 - 1
        i[r.random(i.shape) < 0.05] = -2 ** 31
        return i
    return r.integers(0, E, (T, k))


def _check_rows(torch, dt, T, H, E, k, kind, idx_type="int32", seed=0):
    r = np.random.default_rng(seed)
    idx = _indices(r, T, k, E, kind)
    U.say(f"[tokens {dt}] T={T} H={H} E={E} k={k} {kind}")
    x, fx = U.typed(torch, r.standard_normal((T, H)), dt)
    rows = torch.full((T * k, H), float("nan"), dtype=x.dtype, device="cuda")
    off = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    perm = torch.full((T * k,), -7, dtype=torch.int32, device="cuda")
    inv = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    di = torch.from_numpy(idx).to(getattr(torch, idx_type)).cuda()
    need = qm.qmoe_dispatch_workspace_size(x, di, E)
    qm.qmoe_dispatch(x, di, E, rows, off, perm, inv, torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    rr, ro, rp, ri = S.dispatch(fx, idx, E)
    np.testing.assert_array_equal(off.cpu().numpy(), ro)
    np.testing.assert_array_equal(perm.cpu().numpy(), rp)
    np.testing.assert_array_equal(inv.cpu().numpy(), ri)
    np.testing.assert_array_equal(U.back(rows), rr)
    y, fy = U.typed(torch, r.standard_normal((T * k, H)), dt)
    if ro[-1] < T * k:  # rows of dropped slots are not read
        y[ro[-1]:] = float("nan")
        fy[ro[-1]:] = 0.0
    w = r.standard_normal((T, k)).astype(np.float32)
    dw = torch.from_numpy(w).cuda()
    g, fg = U.typed(torch, r.standard_normal((T, H)), dt)
    gx = torch.full((T, H), float("nan"), dtype=x.dtype, device="cuda")
    out = torch.full_like(gx, float("nan"))
    gr, gw = torch.full_like(y, float("nan")), torch.full_like(dw, float("nan"))
    qm.qmoe_dispatch_backward(y, inv, gx)
    qm.qmoe_combine(y, inv, dw, out)
    qm.qmoe_combine_backward(g, y, inv, dw, gr, gw)
    torch.cuda.synchronize()
    mag = S.combine(np.abs(fy), ri)
    U.check(U.back(gx), S.combine(fy, ri), U.rounded(dt, S.combine(fy, ri), U.sum_bound(k, mag)), "grad_input")
    ref, mag = S.combine(fy, ri, w), S.combine(np.abs(fy), ri, np.abs(w))
    U.check(U.back(out), ref, U.rounded(dt, ref, U.sum_bound(k, mag)), "output")
    rgr, rgw = S.combine_grad(fg, fy, ri, w)
    U.check(U.back(gr), rgr, U.rounded(dt, rgr, 2.0 ** -24 * np.abs(rgr)), "grad_rows")
    _, mag = S.combine_grad(np.abs(fg), np.abs(fy), ri, w)
    U.check(U.back(gw), rgw, U.sum_bound(H, mag) + 2.0 ** -126, "grad_weights")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,H,E,k,kind", [
    (1, 1, 1, 1, "any"), (1, 4096, 8, 2, "any"), (16, 64, 8, 2, "wild"), (3, 17, 5, 3, "wild"), (70, 136, 64, 6, "any"),
    (513, 24, 130, 8, "wild"), (100, 33, 1023, 10, "any"), (9, 2056, 4, 4, "one"), (6, 40, 3, 2, "none"),
    (1100, 9, 7, 4, "one"), (2048, 16, 64, 8, "wild"), (2049, 16, 64, 8, "any")])
def test_rows(torch, dt, T, H, E, k, kind):
    _check_rows(torch, dt, T, H, E, k, kind, "int64" if T % 2 == 0 and kind != "wild" else "int32", seed=T)


def test_rows_int64_indices_beyond_32_bits(torch):
    idx = torch.tensor([[0, 2 ** 32], [2 ** 40 + 1, 1], [-2 ** 33, 1]], device="cuda")
    rows, off, perm, inv = qm.dispatch(torch.ones(3, 4, device="cuda"), idx, 2)
    assert off.tolist() == [0, 1, 3] and perm.tolist() == [0, 3, 5, 1, 2, 4]
    assert inv.tolist() == [[0, -4], [-5, 1], [-6, 2]]
    assert rows[:3].eq(1).all() and rows[3:].eq(0).all()


def test_many_slots_over_many_blocks(torch):
    # 2^20 slots: every block adds up the counts of all others
    r = np.random.default_rng(0)
    T, k, E = 1 << 18, 4, 200
    idx = r.integers(-1, E, (T, k)).astype(np.int32)
    x = torch.arange(T, device="cuda", dtype=torch.float32).view(T, 1).repeat(1, 4)
    rows, off, perm, inv = qm.dispatch(x, torch.from_numpy(idx).cuda(), E)
    flat = np.where(idx.reshape(-1) < 0, E, idx.reshape(-1))
    order = np.argsort(flat, kind="stable")
    np.testing.assert_array_equal(perm.cpu().numpy(), order)
    n = int((flat < E).sum())
    np.testing.assert_array_equal(off.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E + 1))[:E]]))
    got = rows[:, 0].cpu().numpy()
    np.testing.assert_array_equal(got, np.where(np.arange(T * k) < n, order // k, 0))
    place = np.empty(T * k, np.int64)
    place[order] = np.arange(T * k)
    np.testing.assert_array_equal(inv.cpu().numpy().reshape(-1), np.where(flat < E, place, -1 - place))


def test_rows_beyond_two_gib(torch):
    T, H, k, E = 150000, 8192, 2, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    rows, off, perm, inv = qm.dispatch(x, idx, E)
    pick = torch.tensor([0, 5, T - 1, T * k // 2, T * k - 300, T * k - 1], device="cuda")
    assert torch.equal(rows[pick], x[perm[pick].long() // k])
    w = torch.full((T, k), 0.5, device="cuda")
    assert torch.equal(qm.combine(rows, inv, w), x)  # the halves of both copies
    gr, gw = qm.combine_backward(x, rows, inv, w)
    assert torch.equal(gr[pick], (x[perm[pick].long() // k].float() * 0.5).bfloat16())
    tok = torch.tensor([0, T // 2, T - 1], device="cuda")
    ref = (x[tok].double() ** 2).sum(1, keepdim=True).expand(-1, k)
    U.check(U.back(gw[tok]), U.back(ref), U.sum_bound(H, U.back(ref)), "grad_weights")
    assert torch.equal(qm.dispatch_backward(gr, inv), x)


def test_no_tokens_no_slots_no_columns(torch):
    z = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    i = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    rows, off, perm, inv = qm.dispatch(z(0, 8), i(0, 2), 3)
    assert off.tolist() == [0, 0, 0, 0] and rows.shape == (0, 8) and inv.shape == (0, 2)
    assert qm.combine(z(0, 8), i(0, 2), z(0, 2)).shape == (0, 8)
    # tokens without slots: zeros
    rows, off, perm, inv = qm.dispatch(z(5, 8), i(5, 0), 3)
    assert off.tolist() == [0, 0, 0, 0] and rows.shape == (0, 8)
    assert qm.combine(rows, inv, z(5, 0)).eq(0).all()
    # no columns, no experts
    _, off, _, inv = qm.dispatch(z(2, 0), torch.zeros(2, 1, dtype=torch.int32, device="cuda"), 1)
    assert off.tolist() == [0, 2] and inv.tolist() == [[0], [1]]
    gr, gw = qm.combine_backward(z(2, 0), z(2, 0), inv, torch.ones(2, 1, device="cuda"))
    assert gw.eq(0).all()
    rows, off, _, inv = qm.dispatch(torch.ones(2, 4, device="cuda"), torch.zeros(2, 1, dtype=torch.int32, device="cuda"), 0)
    assert off.tolist() == [0] and inv.tolist() == [[-1], [-2]] and rows.eq(0).all()
    idx, w = qm.route(z(0, 4), {"k": 2})
    assert idx.shape == (0, 2)


def test_element_alignment(torch):
    # rows that start off a 16-byte boundary take element accesses
    buf = torch.randn(4 * 64 + 1, device="cuda").half()
    x = buf[1:].view(4, 64)
    idx = torch.tensor([[1], [0], [1], [0]], dtype=torch.int32, device="cuda")
    rows, _, _, inv = qm.dispatch(x, idx, 2)
    assert torch.equal(rows, x[[1, 3, 0, 2]])
    assert torch.equal(qm.combine(rows, inv), x)


# ------------------------------------------------------------------ together
def _layer(torch, c, attrs1, backward=True):
    """A training step of a routed layer with a shared expert, as a user calls it."""
    E = c["w1"].shape[0]
    ra = _attrs(c["k"], "moe", 1)
    idx, w = qm.route(c["logits"], ra)
    rows, off, _, inv = qm.dispatch(c["x"], idx, E)
    h, z = qm.linear(rows, c["w1"], c["b1"], None, off, attrs1, keep_preact=True)
    y = qm.linear(h, c["w2"], c["b2"], None, off)
    routed = qm.combine(y, inv, w)
    hs, zs = qm.linear(c["x"], c["s1"], None, None, None, attrs1, keep_preact=True)
    out = qm.linear(hs, c["s2"], None, routed)  # the shared expert added onto the routed sum
    if not backward:
        return [out]
    g = c["g"]
    ghs, gs2, _ = qm.linear_backward(g, hs, c["s2"])
    gxs, gs1, _ = qm.linear_backward(ghs, c["x"], c["s1"], zs, None, attrs1)
    gy, gw = qm.combine_backward(g, y, inv, w)
    gh, gw2, gb2 = qm.linear_backward(gy, h, c["w2"], None, off, None, bias=True)
    grows, gw1, gb1 = qm.linear_backward(gh, rows, c["w1"], z, off, attrs1, bias=True)
    gx = qm.dispatch_backward(grows, inv)
    gl = qm.route_backward(gw, c["logits"], idx, ra)
    return [out, gx, gxs, gl, gw1, gb1, gw2, gb2, gs1, gs2]


def _layer_case(torch, dt, T, H, E, I, k, seed=0):
    r = np.random.default_rng(seed)
    n = lambda *s, f=1.0: U.typed(torch, r.standard_normal(s) * f, dt)  # noqa: E731
    c, f = {"k": k}, {}
    for name, s, sc in (("x", (T, H), 1), ("w1", (E, 2 * I, H), H ** -0.5), ("b1", (E, 2 * I), 0.1),
                        ("w2", (E, H, I), I ** -0.5), ("b2", (E, H), 0.1), ("s1", (2 * I, H), H ** -0.5),
                        ("s2", (H, I), I ** -0.5), ("g", (T, H), 1)):
        c[name], f[name] = n(*s, f=sc)
    l = r.standard_normal((T, E)).astype(np.float32)
    l[0] = NINF  # a padded token: no expert takes it
    c["logits"], f["logits"] = torch.from_numpy(l).cuda(), l.astype(np.float64)
    return c, f


SWIGLU = {"activation_type": "swiglu", "swiglu_fusion": 1}


def test_layer_in_float32_against_the_oracle(torch):
    T, H, E, I, k = 50, 48, 6, 40, 2
    c, f = _layer_case(torch, "float32", T, H, E, I, k)
    got = [U.back(t) for t in _layer(torch, c, SWIGLU)]
    idx, w = S.route(f["logits"], k, "moe", 1)
    rows, off, _, inv = S.dispatch(f["x"], idx, E)
    h, z = S.linear(rows, f["w1"], f["b1"], None, off, "swiglu")
    y, _ = S.linear(h, f["w2"], f["b2"], None, off)
    hs, zs = S.linear(f["x"], f["s1"], None, None, None, "swiglu")
    out = S.linear(hs, f["s2"], None, S.combine(y, inv, w))[0]
    ghs, gs2, _, _ = S.linear_grad(f["g"], hs, f["s2"])
    gxs, gs1, _, _ = S.linear_grad(ghs, f["x"], f["s1"], zs, None, "swiglu")
    gy, gw = S.combine_grad(f["g"], y, inv, w)
    gh, gw2, gb2, _ = S.linear_grad(gy, h, f["w2"], None, off)
    grows, gw1, gb1, _ = S.linear_grad(gh, rows, f["w1"], z, off, "swiglu")
    ref = [out, S.combine(grows, inv), gxs, S.route_grad(gw, f["logits"], idx, "moe", 1), gw1, gb1, gw2, gb2, gs1, gs2]
    names = ["out", "gx", "gxs", "glogits", "gw1", "gb1", "gw2", "gb2", "gs1", "gs2"]
    for n, a, b in zip(names, got, ref):
        # chained float32 sums of about 100 terms: 100 roundings of 2^-24 a stage, four stages, on the output's scale,
        # with the largest element a few times the RMS
        scale = np.sqrt(np.mean(b ** 2))
        U.check(a, b, np.full(b.shape, 100 * 4 * 4 * 2.0 ** -24) * max(scale, np.abs(b).max()), n)
    assert np.all(got[1][0] == 0) and np.all(got[3][0] == 0)  # the padded token


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_layer_captured_in_a_graph(torch, dt):
    c, _ = _layer_case(torch, dt, 130, 64, 9, 72, 3, seed=1)
    eager = _layer(torch, c, SWIGLU)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _layer(torch, c, SWIGLU)
    for i in range(3):
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        _ = [t.float().sum() for t in eager]  # the program's own work between replays
        torch.cuda.synchronize()
        for p, q in zip(eager, outs):
            assert torch.equal(p, q), i
        # other tokens to other experts, at the same addresses
        c["logits"].copy_(torch.roll(c["logits"], 1, 1))
        c["x"].neg_()
        eager = _layer(torch, c, SWIGLU)


def test_layer_on_a_share_of_the_experts_sums_to_the_whole(torch):
    c, _ = _layer_case(torch, "float32", 60, 32, 8, 24, 3, seed=2)
    idx, w = qm.route(c["logits"], _attrs(3, "qmoe", 0))

    def part(first, held):
        rows, off, _, inv = qm.dispatch(c["x"], idx - first, held)
        h = qm.linear(rows, c["w1"][first:first + held], c["b1"][first:first + held], None, off, SWIGLU)
        return qm.combine(qm.linear(h, c["w2"][first:first + held], c["b2"][first:first + held], None, off), inv, w)
    whole = part(0, 8)
    assert float((part(0, 3) + part(3, 5) - whole).abs().max()) <= 3 * 2.0 ** -23 * float(whole.abs().max())
