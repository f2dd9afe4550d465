"""Pre-activations in 8 bits where only some rows, or none, belong to a group: every row behind the last one, weights of no
groups at all, and large output tiles that end inside groups and in front of a tail."""
import numpy as np
import pytest

import quantized_mixture_experts_router_amd as qm

import front_util as V
import steps_util as U
from test_gpu_linear import attrs_of, make
from test_gpu_linear_q8 import check_forward

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.skip("no GPU")
    return _t


def zero_code(fmt):
    return 128 if fmt == "int8" else 0


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("counts,tail", [([0, 0], 9), ([0], 33), ([], 9), ([], 300)])
def test_rows_of_no_group(torch, dt, counts, tail):
    # (4096: the finishing pass behind a split reduction writes them, where weights have groups)
    for i, (K, N, kind) in enumerate([(40, 72, "swiglu"), (31, 130, "silu"), (64, 256, "gelu"), (4096, 66, "swiglu"), (4096, 33, "relu")]):
        c = make(torch, dt, tail, K, N, counts=counts, kind=kind, residual=i % 2 == 1, seed=i)
        plan = qm.qmoe_linear_plan_describe(c["x"], c["w"], c["off"])
        assert K < 4096 or not plan.startswith(("forward=32x128:1 ", "forward=64x128:1 ")), plan
        fmt, block = ("int8", "e4m3")[i % 2], (128, 32, 64, 16, 128)[i]
        U.say(f"[linear q8 {dt}] {counts}+{tail} {K}->{N} {fmt} {block} {plan}")
        at = attrs_of(kind, {})
        y = torch.full_like(c["dy"], float("nan"))
        codes = torch.full((tail, N), 0x55, dtype=torch.uint8, device="cuda").view(qm._code_type(fmt))
        scales = torch.full((tail, -(-N // block)), float("nan"), device="cuda")
        need = qm.qmoe_linear_q8_workspace_size(c["x"], c["w"], c["b"], c["r"], c["off"], at, y, codes, scales, block)
        ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
        qm.qmoe_linear_q8(c["x"], c["w"], c["b"], c["r"], c["off"], at, y, codes, scales, block, ws)
        assert not y.any() and (scales == 1).all() and (codes.view(torch.uint8) == zero_code(fmt)).all()


@pytest.mark.parametrize("dt", TYPES)
def test_few_rows_in_front_of_a_tail(torch, dt):
    for i, (counts, tail, K, N, kind) in enumerate([([1, 0], 40, 64, 130, "silu"), ([0, 3, 0], 70, 4096, 66, "swiglu"),
                                                    ([2], 31, 4096, 33, "gelu")]):
        c = make(torch, dt, sum(counts) + tail, K, N, counts=counts, kind=kind, residual=i == 1, seed=i)
        check_forward(torch, c, dt, kind, {}, ("int8", "e4m3")[i % 2], (16, 64, 128)[i], f"{counts}+{tail} {K}->{N}")


def scales_of(torch, m, fmt):
    """The least 2^e with m < 127.5 2^e or m <= 464 2^e; 1 for 0."""
    frac, x = torch.frexp(m / (127.5 if fmt == "int8" else 464.0))
    e = x if fmt == "int8" else x - (frac == 0.5).to(x.dtype)
    two = ((e.clamp(min=-126).long() + 1023) << 52).view(torch.float64)  # (ldexp takes a float32 power)
    return torch.where(m == 0, torch.ones_like(m), two)


# counts, tail, K, N, activation: tiles of 256 x 256 in the 16-bit types (128 x 128 or 64 x 128 in float32), ends of groups
# and of columns inside them, columns that allow wide accesses and not
LARGE = [([900, 0, 1173], 127, 64, 4200, "swiglu"), ([257, 1, 700], 42, 64, 8200, "silu"), ([1000, 300, 1], 2, 40, 6201, "gelu"),
         ([2048, 0], 300, 64, 4104, "silu"), ([1500, 1000, 63], 37, 64, 2600, "swiglu")]


@pytest.mark.parametrize("fmt,block", [("int8", 128), ("e4m3", 16)])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("counts,tail,K,N,kind", LARGE)
def test_large_tiles_of_groups(torch, dt, counts, tail, K, N, kind, fmt, block):
    M, live, t = sum(counts) + tail, sum(counts), getattr(torch, dt)
    g = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn(M, K, generator=g, device="cuda").to(t)
    w = (torch.randn(len(counts), N, K, generator=g, device="cuda") / K ** 0.5).to(t)
    b = (torch.randn(len(counts), N, generator=g, device="cuda") * 0.1).to(t)
    ends = np.concatenate([[0], np.cumsum(counts)])
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    plan = qm.qmoe_linear_plan_describe(x, w, off)
    U.say(f"[linear q8 {dt}] {counts}+{tail} {K}->{N} {fmt} {block} {plan}")
    if dt != "float32":
        assert plan.startswith("forward=256x256:1 " if N > 4000 else "forward=128x128:1 "), plan
    at = attrs_of(kind, {})
    y = torch.full((M, N // 2 if kind == "swiglu" else N), float("nan"), dtype=t, device="cuda")
    codes = torch.full((M, N), 0x55, dtype=torch.uint8, device="cuda").view(qm._code_type(fmt))
    scales = torch.full((M, -(-N // block)), float("nan"), device="cuda")
    need = qm.qmoe_linear_q8_workspace_size(x, w, b, None, off, at, y, codes, scales, block)
    ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    qm.qmoe_linear_q8(x, w, b, None, off, at, y, codes, scales, block, ws)
    assert torch.equal(y, qm.linear(x, w, b, None, off, at))
    assert not y[live:].any() and (scales[live:] == 1).all() and (codes[live:].view(torch.uint8) == zero_code(fmt)).all()
    z, A = (torch.zeros(live, N, dtype=torch.float64, device="cuda") for _ in range(2))
    for i, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
        xd, wd, bd = x[lo:hi].double(), w[i].double().t().contiguous(), b[i].double()
        z[lo:hi] = xd @ wd + bd
        A[lo:hi] = xd.abs() @ wd.abs() + bd.abs()
    e = 2.0 * (K + 2) * 2.0 ** -24 * A  # steps_util.sum_bound of K products and the bias
    B = scales.shape[1]
    lo, hi = (torch.zeros(live, B * block, dtype=torch.float64, device="cuda") for _ in range(2))
    lo[:, :N], hi[:, :N] = (z.abs() - e).clamp(min=0), z.abs() + e
    lo, hi = (scales_of(torch, p.view(live, B, block).amax(2), fmt) for p in (lo, hi))
    s = scales[:live].double()
    assert ((s >= lo) & (s <= hi)).all()
    v = qm.dequantize_rows(codes, scales, torch.float32, block)[:live].double()
    step = s.repeat_interleave(block, dim=1)[:, :N]
    half = step / 2 if fmt == "int8" else torch.maximum((z.abs() + e) * 2.0 ** -4, step * 2.0 ** -10)
    assert ((v - z).abs() <= half + e).all()
    if dt == "float32":
        _, zt = qm.linear(x, w, b, None, off, at, keep_preact=True)
        c2, s2 = qm.quantize_rows(zt, fmt, block)
        assert torch.equal(scales, s2) and torch.equal(codes.view(torch.uint8), c2.view(torch.uint8))
