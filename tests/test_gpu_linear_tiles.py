"""Every kind of product of the linear layers (linear_shapes), exactly: inputs
are small integers, so that float32 sums of any order are exact and a result
is the exact one rounded once.  A term left out, taken twice or of another row
shows.  Then an activation of each shape against float64."""
import numpy as np
import pytest

import quantized_mixture_experts_router_amd as qm

import linear_shapes as L
import steps_util as U

pytestmark = pytest.mark.gpu

CASES = [(dt, *s) for dt in ("float32", "float16", "bfloat16") for s in L.SHAPES["float32" if dt == "float32" else "16bit"]]


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.skip("no GPU")
    return _t


def groups_of(M, G, r):
    """Uneven groups (an empty one among five), rows behind the last."""
    if not G:
        return None, M
    share = r.uniform(0.6, 1.4, G)
    if G >= 5:
        share[r.integers(0, G)] = 0.0
    counts = np.floor(share / share.sum() * (M - M // 50 - 1)).astype(int)
    off = np.concatenate([[0], np.cumsum(counts)])
    return off, int(off[-1])


def spans(off, M):
    return [(0, M)] if off is None else list(zip(off[:-1].tolist(), off[1:].tolist()))


def product(torch, a, w, off, turn):
    """Rows of a [M, K] times their group's w ([N, K]: turn, or [K, N]) in float64; rows behind the last group zero."""
    w = w if w.dim() == 3 else w[None]
    out = torch.zeros(a.shape[0], w.shape[1 if turn else 2], dtype=torch.float64, device="cuda")
    for g, (lo, hi) in enumerate(spans(off, a.shape[0])):
        if hi > lo:
            m = w[g].double()
            out[lo:hi] = a[lo:hi].double() @ (m.T if turn else m)
    return out


@pytest.fixture
def ints(torch):
    g = torch.Generator(device="cuda").manual_seed(11)

    def make(t, *shape):
        return torch.randint(-2, 3, shape, generator=g, device="cuda", dtype=torch.int8).to(t)
    return make


def guarded_ws(torch, n):
    return torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dt,M,K,N,G", CASES)
def test_products_exactly(torch, ints, dt, M, K, N, G):
    t = getattr(torch, dt)
    off, live = groups_of(M, G, np.random.default_rng(M + N))
    lead = (G,) if G else ()
    x, w, b = ints(t, M, K), ints(t, *lead, N, K), ints(t, *lead, N)
    r, dy, z = ints(t, M, N), ints(t, M, N), ints(t, M, N)
    for a in (x, r, dy, z):
        a[live:] = float("nan")
    d_off = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    U.say(f"[linear {dt}] {M} x {K} -> {N}, groups {G}: {qm.qmoe_linear_plan_describe(x, w, d_off)}")
    attrs = {"activation_type": "relu"}
    nan = lambda *s: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
    y, kept = nan(M, N), nan(M, N)
    ws = guarded_ws(torch, qm.qmoe_linear_workspace_size(x, w, b, r, d_off, attrs, y, kept))
    qm.qmoe_linear(x, w, b, r, d_off, attrs, y, kept, ws)
    ref = product(torch, x, w, off, True)
    for g, (lo, hi) in enumerate(spans(off, M)):
        ref[lo:hi] += (b if off is None else b[g]).double()
    assert torch.equal(kept, ref.to(t)), "preact"
    ref.clamp_(min=0)
    ref[:live] += r[:live].double()
    assert torch.equal(y, ref.to(t)), "output"
    del y, kept, ref, r
    gx, gw, gb = nan(M, K), nan(*lead, N, K), nan(*lead, N)
    ws = guarded_ws(torch, qm.qmoe_linear_backward_workspace_size(dy, x, w, z, d_off, attrs, gx, gw, gb))
    qm.qmoe_linear_backward(dy, x, w, z, d_off, attrs, gx, gw, gb, ws)
    d = torch.where(z > 0, dy, torch.zeros_like(dy))
    assert torch.equal(gx, product(torch, d, w, off, False).to(t)), "grad_input"
    for g, (lo, hi) in enumerate(spans(off, M)):
        f = d[lo:hi].double()
        assert torch.equal(gw[g] if G else gw, (f.T @ x[lo:hi].double()).to(t)), f"grad_weights of group {g}"
        assert torch.equal(gb[g] if G else gb, f.sum(0).to(t)), f"grad_bias of group {g}"


ACTS = [("gelu", {}), ("swiglu", {}), ("silu", {}), ("swiglu", dict(alpha=1.7, beta=0.5, limit=0.8))]


@pytest.mark.parametrize("dt,M,K,N,G", CASES)
def test_epilogues(torch, dt, M, K, N, G):
    # float64 on the GPU; the bounds are steps_util's
    i = CASES.index((dt, M, K, N, G))
    kind, a = ACTS[i % 4]
    t = getattr(torch, dt)
    gen = torch.Generator(device="cuda").manual_seed(i)
    off, live = groups_of(M, G, np.random.default_rng(M + N))
    lead = (G,) if G else ()
    rnd = lambda s, *shape: (torch.randn(*shape, generator=gen, device="cuda") * s).to(t)  # noqa: E731
    x, w, b = rnd(1, M, K), rnd(K ** -0.5, *lead, N, K), rnd(0.1, *lead, N)
    No = N // 2 if kind == "swiglu" else N
    r = rnd(1, M, No) if i % 3 else None
    d_off = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    attrs = {"activation_type": kind, "swiglu_fusion": int(kind == "swiglu")}
    if a:
        attrs.update(activation_alpha=a["alpha"], activation_beta=a["beta"], swiglu_limit=a["limit"])
    U.say(f"[linear {dt}] {M} x {K} -> {N}, groups {G}, {kind} {a}")
    y = qm.linear(x, w, b, r, d_off, attrs)
    z, A = product(torch, x, w, off, True), product(torch, x.abs(), w.abs(), off, True)
    for g, (lo, hi) in enumerate(spans(off, M)):
        bg = (b if off is None else b[g]).double()
        z[lo:hi] += bg
        A[lo:hi] += bg.abs()
    ez = 2.0 * (K + 1) * 2.0 ** -24 * A
    al, be = a.get("alpha", 1.0), a.get("beta", 0.0)
    if kind == "gelu":
        ref, e = z * torch.special.ndtr(z), 1.13 * ez + U.EV * z.abs()
    elif kind == "silu":
        ref, e = z * torch.sigmoid(z), 1.13 * ez + U.EV * z.abs()
    else:
        p, u = z[:, 0::2], z[:, 1::2]
        ep, eu = ez[:, 0::2], ez[:, 1::2]
        if "limit" in a:
            p, u = p.clamp(max=a["limit"]), u.clamp(-a["limit"], a["limit"])
        ref = p * torch.sigmoid(al * p) * (u + be)
        e = 1.1 * ((u + be).abs() + eu) * ep + (p.abs() + ep) * eu + U.EV * p.abs() * (u.abs() + abs(be))
    if r is not None:
        ref[:live] += r[:live].double()
        e[:live] += 2.0 ** -23 * (ref[:live].abs() + r[:live].double().abs() + e[:live])
    ref[live:] = 0
    bound = U.HALF[dt] * (ref.abs() + e) + U.TINY[dt] + e
    bound[live:] = 0
    err = (y.double() - ref).abs()
    assert not torch.isnan(err).any()
    U.say(f"  output: max err / bound = {float((err[:live] / bound[:live]).max()):.3g}")
    assert bool((err <= bound).all())


# the large tile of each type in every product (float32: a shape a product)
LARGE = [("bfloat16", 3000, 3336, 4104, "forward=256x256:1 grad_input=256x256:1 grad_weights=256x256:1"),
         ("float16", 3000, 3336, 4104, "forward=256x256:1 grad_input=256x256:1 grad_weights=256x256:1"),
         ("float32", 5378, 168, 1286, "forward=128x128:1"), ("float32", 4125, 1864, 168, "grad_input=128x128:1"),
         ("float32", 169, 1587, 4792, "grad_weights=128x128:1")]


def large(torch, dt, M, K, N, tiles):
    t = getattr(torch, dt)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, w = torch.randn(M, K, generator=g, device="cuda").to(t), torch.randn(N, K, generator=g, device="cuda").to(t)
    plan = qm.qmoe_linear_plan_describe(x, w)
    assert tiles in plan, plan
    U.say(f"[linear {dt}] {M} x {K} -> {N}: {plan}")
    return t, g, x, w


@pytest.mark.parametrize("dt,M,K,N,tiles", LARGE)
def test_large_tiles_keep_infinities_in_their_row_and_column(torch, dt, M, K, N, tiles):
    t, g, x, w = large(torch, dt, M, K, N, tiles)
    dy = torch.randn(M, N, generator=g, device="cuda").to(t)
    x[M - 1, K - 3], w[150, 9], dy[130, N - 2] = float("inf"), float("nan"), float("-inf")
    y = qm.linear(x, w)
    gx, gw, gb = qm.linear_backward(dy, x, w, bias=True)

    def only(a, row, col):
        want = torch.zeros_like(a, dtype=torch.bool)
        want[row] = True
        want[:, col] = True
        assert torch.equal(~torch.isfinite(a), want)
    only(y, M - 1, 150)
    only(gx, 130, 9)
    only(gw, N - 2, K - 3)
    assert not torch.isfinite(gb[N - 2]) and torch.isfinite(gb).sum() == N - 1


@pytest.mark.parametrize("dt,M,K,N,tiles", LARGE)
def test_large_tiles_in_a_graph(torch, dt, M, K, N, tiles):
    t, g, x, w = large(torch, dt, M, K, N, tiles)
    dy, z = torch.randn(M, N, generator=g, device="cuda").to(t), torch.randn(M, N, generator=g, device="cuda").to(t)
    a = {"activation_type": "silu"}
    call = lambda: [qm.linear(x, w, None, dy, None, a), *qm.linear_backward(dy, x, w, z, None, a, bias=True)]  # noqa: E731
    eager = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for i in range(3):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        _ = [o.float().sum() for o in eager]  # the program's own work between replays
        torch.cuda.synchronize()
        for p, q in zip(eager, outs):
            assert torch.equal(p, q), i
        x.neg_()
        eager = call()


@pytest.mark.parametrize("dt,M,K,N,tiles", [
    ("bfloat16", 3000, 3333, 4106, "forward=256x256:1 grad_input=256x256:1 grad_weights=256x256:1"),
    ("float32", 5379, 169, 1286, "forward=128x128:1"), ("float32", 4125, 1863, 166, "grad_input=128x128:1"),
    ("float32", 169, 1587, 4790, "grad_weights=128x128:1")])
def test_large_tiles_of_element_aligned_tensors(torch, ints, dt, M, K, N, tiles):
    # rows of no whole 16-byte runs at odd addresses: padded operands, single stores
    t = getattr(torch, dt)

    def odd(*shape):
        n = int(np.prod(shape))
        v = torch.empty(n + 1, dtype=t, device="cuda")[1:].view(shape)
        return v.copy_(ints(t, *shape))
    x, w, b, dy = odd(M, K), odd(N, K), odd(N), odd(M, N)
    U.say(f"[linear {dt}] {M} x {K} -> {N}: {qm.qmoe_linear_plan_describe(x, w)}")
    assert tiles in qm.qmoe_linear_plan_describe(x, w)
    y = qm.linear(x, w, b, dy)
    assert torch.equal(y, (product(torch, x, w, None, True) + b.double() + dy.double()).to(t))
    gx, gw, gb = qm.linear_backward(dy, x, w, bias=True)
    assert torch.equal(gx, product(torch, dy, w, None, False).to(t))
    assert torch.equal(gw, (dy.double().T @ x.double()).to(t))
    assert torch.equal(gb, dy.double().sum(0).to(t))


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("G", [63, 64, 65, 127, 128, 129, 1023])
def test_many_groups(torch, ints, dt, G):
    # the walk over groups goes 64 at a time; the first offset is taken as 0
    t = getattr(torch, dt)
    r = np.random.default_rng(G)
    counts = r.integers(0, 9, G) * (r.random(G) < 0.7)
    counts[G - 1], counts[G // 2] = 70, 150
    off = np.concatenate([[0], np.cumsum(counts)])
    M, K, N = int(off[-1]) + 33, 72, 136
    x, w, b, dy, z = ints(t, M, K), ints(t, G, N, K), ints(t, G, N), ints(t, M, N), ints(t, M, N)
    first = int(off[1]) if off[1] else 0
    given = off.copy()
    given[0] = first // 2
    d_off = torch.tensor(given, dtype=torch.int32, device="cuda")
    U.say(f"[linear {dt}] {M} rows in {G} groups: {qm.qmoe_linear_plan_describe(x, w, d_off)}")
    a = {"activation_type": "relu"}
    y = qm.linear(x, w, b, None, d_off, a)
    ref = product(torch, x, w, off, True)
    for g, (lo, hi) in enumerate(spans(off, M)):
        ref[lo:hi] += b[g].double()
    assert torch.equal(y, ref.clamp(min=0).to(t))
    gx, gw, gb = qm.linear_backward(dy, x, w, z, d_off, a, bias=True)
    d = torch.where(z > 0, dy, torch.zeros_like(dy))
    assert torch.equal(gx, product(torch, d, w, off, False).to(t))
    for g, (lo, hi) in enumerate(spans(off, M)):
        f = d[lo:hi].double()
        assert torch.equal(gw[g], (f.T @ x[lo:hi].double()).to(t)), g
        assert torch.equal(gb[g], f.sum(0).to(t)), g
