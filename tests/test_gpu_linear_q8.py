"""Linear layers that leave their pre-activations in 8 bits, and their gradients
from what is held in 8 bits.  The output has qmoe_linear's bits; the 8-bit rows
are held to the float64 oracle's pre-activations and, in float32, to the rows
that qmoe_quantize_rows makes of qmoe_linear's; gradients have the bits of
qmoe_linear_backward on the values that the codes stand for."""
import numpy as np
import pytest

import quantized_mixture_experts_router_amd as qm
from oracle import steps_oracle as S

import front_util as V
import steps_util as U
from test_gpu_linear import ACTS, attrs_of, make, ws_of

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.skip("no GPU")
    return _t


def check_forward(torch, c, dt, kind, a, fmt, block, label):
    U.say(f"[linear q8 {dt}] {label} {kind} {fmt} {block}")
    at = attrs_of(kind, a)
    M, N = c["x"].shape[0], c["w"].shape[-2]
    y = torch.full_like(c["dy"], float("nan"))
    codes = torch.full((M, N), 0x55, dtype=torch.uint8, device="cuda").view(qm._code_type(fmt))
    scales = torch.full((M, -(-N // block)), float("nan"), device="cuda")
    need = qm.qmoe_linear_q8_workspace_size(c["x"], c["w"], c["b"], c["r"], c["off"], at, y, codes, scales, block)
    qm.qmoe_linear_q8(c["x"], c["w"], c["b"], c["r"], c["off"], at, y, codes, scales, block, ws_of(torch, need))
    torch.cuda.synchronize()
    assert torch.equal(y, qm.linear(c["x"], c["w"], c["b"], c["r"], c["off"], at))
    _, rz = S.linear(c["fx"], c["fw"], c["fb"], c["fr"], c["foff"], kind, **a)
    A = S.preact(np.abs(c["fx"]), np.abs(c["fw"]), None if c["fb"] is None else np.abs(c["fb"]), c["foff"])
    V.check_eight(torch, codes, scales, block, rz, U.sum_bound(c["fx"].shape[1], A), "preact")
    n = S.live_rows(M, c["fw"], c["foff"])
    assert (scales[n:] == 1).all() and (codes[n:].view(torch.uint8) == (128 if fmt == "int8" else 0)).all()
    if dt == "float32":
        _, z = qm.linear(c["x"], c["w"], c["b"], c["r"], c["off"], at, keep_preact=True)
        c2, s2 = qm.quantize_rows(z, fmt, block)
        assert torch.equal(scales, s2) and torch.equal(codes.view(torch.uint8), c2.view(torch.uint8))
    out = qm.linear_q8(c["x"], c["w"], c["b"], c["r"], c["off"], at, fmt, block)
    assert torch.equal(out[0], y) and torch.equal(out[1].view(torch.uint8), codes.view(torch.uint8)) and torch.equal(out[2], scales)


SIZES = [(1, 8, 8), (3, 40, 24), (7, 33, 20), (33, 64, 130), (130, 96, 264), (65, 1024, 31), (300, 72, 129)]


@pytest.mark.parametrize("kind,a", ACTS)
@pytest.mark.parametrize("dt", TYPES)
def test_forward(torch, dt, kind, a):
    for i, (M, K, N) in enumerate(SIZES):
        N += N % 2 if kind == "swiglu" else 0
        c = make(torch, dt, M, K, N, kind=kind, bias=i % 2 == 0, residual=i % 3 == 0, seed=i)
        check_forward(torch, c, dt, kind, a, ("int8", "e4m3")[i % 2], V.BLOCKS[i % 4], f"{M}x{K}->{N}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("counts,tail", [([5, 0, 70, 1], 0), ([0, 0, 33], 7), ([], 9), ([130, 2], 40)])
def test_forward_of_groups(torch, dt, counts, tail):
    for i, (K, N, kind) in enumerate([(40, 72, "swiglu"), (31, 130, "silu"), (64, 256, "gelu")]):
        if not counts:
            continue
        c = make(torch, dt, sum(counts) + tail, K, N, counts=counts, kind=kind, residual=i == 1, seed=i)
        check_forward(torch, c, dt, kind, {}, ("int8", "e4m3")[i % 2], (128, 32, 64)[i], f"{counts}+{tail} {K}->{N}")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,K,N,G", [(1, 4096, 40, 0), (5, 8192, 130, 0), (40, 4096, 33, 0), (9, 4096, 66, 3)])
def test_forward_of_split_reductions(torch, dt, M, K, N, G):
    counts = [M - 4, 0, 2] if G else None
    c = make(torch, dt, M, K, N, counts=counts, kind="silu", seed=M)
    plan = qm.qmoe_linear_plan_describe(c["x"], c["w"], c["off"])
    assert not plan.startswith(("forward=32x128:1 ", "forward=64x128:1 ")), plan
    check_forward(torch, c, dt, "silu", {}, "int8", 16, plan)
    check_forward(torch, c, dt, "silu", {}, "e4m3", 128, plan)


@pytest.mark.parametrize("dt", TYPES)
def test_forward_of_large_tiles(torch, dt):
    c = make(torch, dt, 520, 64, 4200, kind="swiglu", seed=1)
    check_forward(torch, c, dt, "swiglu", {}, "int8", 128, qm.qmoe_linear_plan_describe(c["x"], c["w"]))
    for M, N in ((4096, 4096), (2048, 2050)):  # against quantize_rows of the float32 layer's; 16-bit types by their plans
        g = torch.Generator(device="cuda").manual_seed(M)
        x = torch.randn(M, 40, generator=g, device="cuda").to(getattr(torch, dt))
        w = (torch.randn(N, 40, generator=g, device="cuda") / 6).to(x.dtype)
        U.say(f"[linear q8 {dt}] {M} x {N}: {qm.qmoe_linear_plan_describe(x, w)}")
        y, codes, scales = qm.linear_q8(x, w, attrs={"activation_type": "silu"})
        assert torch.equal(y, qm.linear(x, w, attrs={"activation_type": "silu"}))
        z = x.double() @ w.double().t()
        m = torch.zeros(M, -(-N // 128) * 128, dtype=torch.float64, device="cuda")
        m[:, :N] = z.abs()
        m = m.view(M, -1, 128).amax(2)
        e = 2 * 41 * 2.0 ** -24 * (x.double().abs() @ w.double().abs().t())
        # the scale: m (1 +- e) lies between 63.5 and 127.5 scales (a border passed: the other one)
        assert ((m >= scales.double() * 63.75 * (1 - 1e-4)) & (m < scales.double() * 127.5 * (1 + 1e-4))).all()
        step = scales.double().repeat_interleave(128, dim=1)[:, :N]
        v = qm.dequantize_rows(codes, scales, torch.float32).double()
        assert ((v - z).abs() <= step / 2 + e).all()


# ------------------------------------------------------------------ gradients
def bits(torch, t):
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def check_backward(torch, c, dt, kind, a, fmt, block, k=0, x8=True, z8=True, which=(True, True, True), seed=0):
    U.say(f"[linear grad q8 {dt}] {tuple(c['x'].shape)} -> {c['w'].shape[-2]} {kind} {fmt} {block} k={k} {x8} {z8}")
    at = attrs_of(kind, a)
    x, z, perm = c["x"], c["z"], None
    M = x.shape[0]
    if k:
        x = x[:M // k].contiguous()
        perm = torch.randperm(M, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    hx, hz = x, z
    if x8:
        hx = qm.quantize_rows(x, fmt, block)
        x = qm.dequantize_rows(*hx, x.dtype, block, perm=perm)
    if z8 and z is not None:
        hz = qm.quantize_rows(z, ("e4m3", "int8")[fmt == "e4m3"], block)
        z = qm.dequantize_rows(*hz, z.dtype, block)
    want = qm.linear_backward(c["dy"], x, c["w"], z, c["off"], at, bias=True)
    got = qm.linear_backward_q8(c["dy"], hx, c["w"], hz, c["off"], at, True, block, perm)
    for g, r, name in zip(got, want, ("grad_input", "grad_weights", "grad_bias")):
        assert torch.equal(bits(torch, g), bits(torch, r)), name
    # each alone, in a workspace of its own size
    for i in range(3):
        only = [torch.full_like(g, float("nan")) if j == i else None for j, g in enumerate(want)]
        need = qm.qmoe_linear_backward_q8_workspace_size(c["dy"], hx, c["w"], hz, c["off"], at, *only, block, perm)
        qm.qmoe_linear_backward_q8(c["dy"], hx, c["w"], hz, c["off"], at, *only, block, perm, ws_of(torch, need))
        assert torch.equal(bits(torch, only[i]), bits(torch, want[i])), i


@pytest.mark.parametrize("kind,a", ACTS)
@pytest.mark.parametrize("dt", TYPES)
def test_backward(torch, dt, kind, a):
    for i, (M, K, N) in enumerate(SIZES):
        N += N % 2 if kind == "swiglu" else 0
        c = make(torch, dt, M, K, N, kind=kind, seed=i)
        check_backward(torch, c, dt, kind, a, ("int8", "e4m3")[i % 2], V.BLOCKS[i % 4], x8=i != 4, z8=i != 5)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("counts,tail,k", [([5, 0, 70, 1], 0, 4), ([0, 0, 33], 7, 5), ([130, 2], 40, 0), ([12], 0, 12)])
def test_backward_of_groups(torch, dt, counts, tail, k):
    for i, (K, N, kind) in enumerate([(40, 72, "swiglu"), (31, 130, "silu"), (64, 256, "identity"), (129, 33, "relu")]):
        c = make(torch, dt, sum(counts) + tail, K, N, counts=counts, kind=kind, seed=i)
        check_backward(torch, c, dt, kind, {}, ("int8", "e4m3")[i % 2], (128, 32, 64, 16)[i], k, seed=i)


def test_backward_against_the_definition(torch):
    # gradients from 8 bits against the oracle's on the stored values (float32: per element as the other gradients)
    c = make(torch, "float32", 24, 40, 36, counts=[3, 0, 15], kind="silu", seed=2)
    hx, hz = qm.quantize_rows(c["x"], "int8", 32), qm.quantize_rows(c["z"], "e4m3", 32)
    fx, fz = V.stored(torch, *hx, 32), V.stored(torch, *hz, 32)
    gi, gw, gb = qm.linear_backward_q8(c["dy"], hx, c["w"], hz, c["off"], attrs_of("silu", {}), True, 32)
    dx, dw, db, d = S.linear_grad(c["fdy"], fx, c["fw"], fz, c["foff"], "silu")
    ed = U.grad_eval_bound(c["fdy"], fz, "silu") + 2.0 ** -24 * np.abs(d)
    ax, aw, ab, _ = S.linear_grad(np.abs(d) + ed, np.abs(fx), np.abs(c["fw"]), None, c["foff"])
    ex, ew, eb, _ = S.linear_grad(ed, np.abs(fx), np.abs(c["fw"]), None, c["foff"])
    for got, ref, A, e, n in ((gi, dx, ax, ex, 36), (gw, dw, aw, ew, 24), (gb, db, ab, eb, 24)):
        U.check(U.back(got), ref, U.rounded("float32", ref, U.sum_bound(n, A) + e), "gradient")


def test_what_is_not_finite_stays_in_its_rows(torch):
    c = make(torch, "bfloat16", 20, 32, 48, kind="silu", seed=3)
    z = c["z"].clone()
    z[4, 5] = float("inf")
    hz = qm.quantize_rows(z, "int8", 16)
    gi, gw, _ = qm.linear_backward_q8(c["dy"], c["x"], c["w"], hz, None, attrs_of("silu", {}), True, 16)
    assert gi[4].isnan().all()
    rest = torch.arange(20, device="cuda") != 4
    assert gi[rest].isfinite().all()
    assert gw[:16].isnan().all() and gw[16:].isfinite().all()  # the block's columns


def test_empty(torch):
    x, w = torch.zeros(0, 8, device="cuda"), torch.ones(4, 8, device="cuda")
    y, c, s = qm.linear_q8(x, w)
    assert y.shape == (0, 4) and c.shape == (0, 4) and s.shape == (0, 1)
    gi, gw, gb = qm.linear_backward_q8(y, qm.quantize_rows(x), w, (c, s), attrs={"activation_type": "relu"}, bias=True)
    assert gi.shape == (0, 8) and not gw.any() and not gb.any()
