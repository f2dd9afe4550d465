"""The norm, routing from scores, dispatch, experts and combine as a training
step uses them, with 8-bit checkpoints: against the float64 oracle, captured in
graphs, on streams of their own and from two calls at once."""
import numpy as np
import pytest

import quantized_mixture_experts_router_amd as qm
from oracle import front_oracle as F
from oracle import steps_oracle as S

import front_util as V
import steps_util as U

pytestmark = pytest.mark.gpu

T, H, I, E, K = 37, 64, 48, 8, 3
ROUTE = {"k": K, "scores": "sigmoid", "groups": 4, "kept_groups": 2, "normalize_routing_weights": 1, "scale": 2.5}
ACT = {"activation_type": "swiglu", "swiglu_fusion": 1}


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.skip("no GPU")
    return _t


def inputs(torch, dt, seed=0):
    r = np.random.default_rng(seed)
    f = {"x": r.standard_normal((T, H)), "r": r.standard_normal((T, H)), "g": 1 + 0.1 * r.standard_normal(H),
         "wr": r.standard_normal((E, H)) / H ** 0.5, "w1": r.standard_normal((E, 2 * I, H)) / H ** 0.5,
         "w2": r.standard_normal((E, H, I)) / I ** 0.5, "dy": r.standard_normal((T, H)), "ds": r.standard_normal((T, H))}
    t = {k: torch.from_numpy(v).to(getattr(torch, dt)).cuda() for k, v in f.items()}
    t["b"] = torch.from_numpy(r.standard_normal(E) * 0.05).float().cuda()
    return t


def step(t):
    """Forward and backward of one layer: every result, in order."""
    y, h, y8, ys = qm.rms_norm(t["x"], t["g"], t["r"], format="int8", block_size=32)
    logits = qm.linear(y, t["wr"]).float()
    idx, w = qm.route_scored(logits, t["b"], ROUTE)
    rows, off, perm, inv = qm.dispatch(y, idx, E)
    a, z8, zs = qm.linear_q8(rows, t["w1"], None, None, off, ACT, "e4m3", 32)
    o = qm.linear(a, t["w2"], offsets=off)
    out = qm.combine(o, inv, w)
    do, dw = qm.combine_backward(t["dy"], o, inv, w)
    da, dw2, _ = qm.linear_backward(do, a, t["w2"], offsets=off)
    drows, dw1, _ = qm.linear_backward_q8(da, (y8, ys), t["w1"], (z8, zs), off, ACT, block_size=32, perm=perm)
    dl = qm.route_scored_backward(dw, logits, idx, ROUTE)
    dyr, dwr, _ = qm.linear_backward_q8(dl.to(y.dtype), (y8, ys), t["wr"], block_size=32)
    dyn = qm.dispatch_backward(drows, inv) + dyr
    dx, dg = qm.rms_norm_backward(dyn, h, t["g"], t["ds"])
    return [out, h, y8.view(y8.dtype), ys, idx, w, z8, zs, dw1, dw2, dwr, dl, dx, dg]


def same(torch, a, b):
    def raw(t):
        return t.contiguous().view(torch.uint8)
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(raw(x), raw(y)), i


def test_step_against_the_definition(torch):
    t = inputs(torch, "float32")
    out, h, y8, ys, idx, w, z8, zs, dw1, dw2, dwr, dl, dx, dg = step(t)
    torch.cuda.synchronize()
    f = {k: v.double().cpu().numpy() for k, v in t.items()}
    fh = (t["x"].cpu() + t["r"].cpu()).double().numpy()
    y = F.rms_norm(fh, f["g"])
    logits = y @ f["wr"].T
    ri, rw = F.route_scored(logits, K, "sigmoid", f["b"], 4, 2, 2, 1, 2.5)
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    rows, off, perm, inv = S.dispatch(y, ri, E)
    a, z = S.linear(rows, f["w1"], None, None, off, "swiglu")
    o, _ = S.linear(a, f["w2"], None, None, off)
    ro = S.combine(o, inv, rw)
    # what the checkpoints hold stands for the rows and pre-activations in the backward pass
    hy, hz = V.stored(torch, y8, ys, 32), V.stored(torch, z8, zs, 32)
    do, dw = S.combine_grad(f["dy"], o, inv, rw)
    da, rw2, _, _ = S.linear_grad(do, a, f["w2"], None, off)
    drows, rw1, _, _ = S.linear_grad(da, F.slots(hy, perm, K), f["w1"], hz, off, "swiglu")
    rl = F.route_scored_grad(dw, logits, ri, "sigmoid", 1, 2.5)
    dyr, rwr, _, _ = S.linear_grad(rl, hy, f["wr"])
    rx, rg = F.rms_norm_grad(S.combine(drows, inv) + dyr, fh, f["g"], f["ds"])
    # seven float32 sums of at most 96 terms lie behind any result, each within 2 x 97 x 2^-24 of its magnitudes, which are
    # below 8 times their result's norm (normal operands: sqrt(96) at most, less one factor in the mean): 2^-10
    for got, ref, name in ((out, ro, "out"), (w, rw, "w"), (dw1, rw1, "dw1"), (dw2, rw2, "dw2"), (dwr, rwr, "dwr"), (dl, rl, "dl"),
                           (dx, rx, "dx"), (dg, rg, "dg")):
        rel = np.linalg.norm(U.back(got) - ref) / np.linalg.norm(ref)
        U.say(f"  {name}: {rel:.2e}")
        assert rel <= 2.0 ** -10, name
    # 8 bits in the place of the rows themselves change the gradients by no more than the format's rounding: half a step is
    # 2^-4 of a value at most (e4m3, z) and 1 / 127 of a block's largest (int8, y); measured against the oracle without them
    dr, full1, _, _ = S.linear_grad(da, rows, f["w1"], z, off, "swiglu")
    rel = np.linalg.norm(rw1 - full1) / np.linalg.norm(full1)
    assert 0 < rel < 2.0 ** -3, rel


@pytest.mark.parametrize("dt", ["float32", "float16", "bfloat16"])
def test_step_repeats_and_replays(torch, dt):
    t = inputs(torch, dt, 1)
    want = step(t)
    same(torch, step(t), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(t)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(t)
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        same(torch, got, want)
        same(torch, step(t), want)  # eager work between the replays
    # new values in the same buffers
    u = inputs(torch, dt, 2)
    for k in t:
        t[k].copy_(u[k])
    graph.replay()
    torch.cuda.synchronize()
    same(torch, got, step(u))


def test_two_graphs_and_a_stream_at_once(torch):
    ts = [inputs(torch, "bfloat16", s) for s in (3, 4, 5)]
    want = [step(t) for t in ts]
    torch.cuda.synchronize()
    graphs, got = [], []
    for t in ts[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(step(t))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            last = step(ts[2])
        torch.cuda.synchronize()
        same(torch, got[0], want[0])
        same(torch, got[1], want[1])
        same(torch, last, want[2])


def test_calls_on_a_given_stream(torch):
    t = inputs(torch, "float16", 6)
    s = torch.cuda.Stream()
    want = qm.rms_norm(t["x"], t["g"], t["r"], format="int8")
    torch.cuda.synchronize()
    got = qm.rms_norm(t["x"], t["g"], t["r"], format="int8", stream=s)
    logits = torch.randn(9, 8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    i, w = qm.route_scored(logits, None, {"k": 2}, stream=s)
    c, sc = qm.quantize_rows(t["x"], "e4m3", 16, stream=s)
    v = qm.dequantize_rows(c, sc, torch.float16, 16, stream=s)
    gx, gw = qm.rms_norm_backward(t["dy"], t["x"], t["g"], stream=s)
    y, z, zs = qm.linear_q8(t["x"], t["wr"], stream=s)
    gi, gww, _ = qm.linear_backward_q8(y, (c, sc), t["wr"], block_size=16, stream=s)
    s.synchronize()
    same(torch, got, want)
    same(torch, (i, w), qm.route_scored(logits, None, {"k": 2}))
    same(torch, (v, gx, gw), (qm.dequantize_rows(c, sc, torch.float16, 16), *qm.rms_norm_backward(t["dy"], t["x"], t["g"])))
    same(torch, (y, z, zs), qm.linear_q8(t["x"], t["wr"]))
    same(torch, (gi, gww), qm.linear_backward_q8(y, (c, sc), t["wr"], block_size=16)[:2])
