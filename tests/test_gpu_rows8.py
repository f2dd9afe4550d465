"""GPU parity of rows in 8 bits: scales, codes and values equal the oracle's
(both directions are exact but for the one rounding that the format defines)."""
import numpy as np
import pytest

import quantized_mixture_experts_router_amd as qm
from oracle import front_oracle as F

import front_util as V
import steps_util as U

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]
FORMATS = ["int8", "e4m3"]


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.skip("no GPU")
    return _t


def check(torch, x, fmt, block, dt):
    U.say(f"[rows8] {tuple(x.shape)} {dt} {fmt} block {block}")
    codes, scales = qm.quantize_rows(x, fmt, block)
    torch.cuda.synchronize()
    ref, s = F.eight(x.double().cpu().numpy(), fmt, block)
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    got = V.stored(torch, codes, scales, block)
    np.testing.assert_array_equal(got, ref)
    for out in TYPES:
        t = getattr(torch, out)
        top = torch.finfo(t).max
        want = torch.from_numpy(ref).clamp(-top, top).to(t)
        val = qm.dequantize_rows(codes, scales, t, block)
        assert val.dtype == t
        assert torch.equal(val.cpu().nan_to_num(7.0), want.nan_to_num(7.0)), out
        assert torch.equal(val.cpu().isnan(), want.isnan()), out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,N,block", [(1, 1, 16), (3, 7, 16), (5, 16, 16), (2, 33, 32), (9, 129, 64), (4, 128, 128),
                                       (17, 260, 128), (1, 1000, 32), (33, 72, 16), (7, 2049, 128)])
def test_rows(torch, dt, fmt, M, N, block):
    r = np.random.default_rng(M * N + block)
    x = r.standard_normal((M, N)) * np.exp(2 * r.standard_normal(N))
    check(torch, torch.from_numpy(x).to(getattr(torch, dt)).cuda(), fmt, block, dt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", TYPES)
def test_borders(torch, dt, fmt):
    # largest magnitudes on either side of where the scale grows, halves of a step, zeros, the type's ends, and what is
    # not finite, a block of 16 each
    t = getattr(torch, dt)
    f = torch.finfo(t)
    tops = [127.0, 127.5, 127.4375, 128.0, 255.0, 464.0, 448.0, 465.0, 1.0, 0.0, f.max, -f.max, f.tiny, f.smallest_normal * f.eps,
            float("inf"), float("-inf"), float("nan"), 2.0 ** -14, 3.0]
    rows = []
    for top in tops:
        fill = [0.5, 1.5, 2.5, -3.5, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 0.0, -0.0, 7.5, 17.0, 19.0, 25.0, -27.0, 0.03125]
        k = abs(top) / 464.0 if np.isfinite(top) and 0 < abs(top) < 1e-3 else 1.0
        fill = [v * k if np.isfinite(top) and abs(top) != 0.0 and abs(top) < 1e-3 else min(abs(top), abs(v)) if np.isfinite(top) else v for v in fill]
        rows.append([top] + fill)
    x = torch.tensor(rows, dtype=torch.float64).to(t).cuda()
    check(torch, x, fmt, 16, dt)
    check(torch, x.reshape(1, -1).contiguous(), fmt, 16, dt)


@pytest.mark.parametrize("offset", [1, 3])
@pytest.mark.parametrize("N", [40, 129])
def test_any_element_alignment(torch, N, offset):
    r = np.random.default_rng(offset)
    base = torch.from_numpy(r.standard_normal(6 * N + 8)).bfloat16().cuda()
    x = base[offset:offset + 6 * N].view(6, N)
    c = torch.full((6 * N + 8,), 77, dtype=torch.uint8, device="cuda")
    s = torch.empty(6, -(-N // 32), device="cuda")
    qm.qmoe_quantize_rows(x, 32, c[offset:offset + 6 * N].view(6, N), s)
    ref, rs = F.eight(x.double().cpu().numpy(), "int8", 32)
    np.testing.assert_array_equal(V.stored(torch, c[offset:offset + 6 * N].view(6, N), s, 32), ref)
    assert (c[:offset] == 77).all() and (c[offset + 6 * N:] == 77).all()
    out = torch.full((6 * N + 8,), 5.0, dtype=torch.float16, device="cuda")
    o = out[offset:offset + 6 * N].view(6, N)
    qm.qmoe_dequantize_rows(c[offset:offset + 6 * N].view(6, N), s, 32, None, o)
    np.testing.assert_array_equal(U.back(o), ref.astype(np.float16).astype(np.float64))
    assert (out[:offset] == 5).all() and (out[offset + 6 * N:] == 5).all()


@pytest.mark.parametrize("dt,fmt", [("float32", "int8"), ("float16", "e4m3"), ("bfloat16", "int8")])
@pytest.mark.parametrize("T,k,N", [(5, 1, 40), (7, 3, 129), (64, 6, 256), (1, 8, 8)])
def test_tokens_rows_to_slots(torch, dt, fmt, T, k, N):
    r = np.random.default_rng(T * k)
    x = torch.from_numpy(r.standard_normal((T, N))).to(getattr(torch, dt)).cuda()
    idx = torch.from_numpy(r.integers(-1, 4, (T, k)).astype(np.int32)).cuda()
    rows, off, perm, inv = qm.dispatch(x, idx, 4)
    codes, scales = qm.quantize_rows(x, fmt, 64)
    got = qm.dequantize_rows(codes, scales, x.dtype, 64, perm=perm)
    ref = F.slots(V.stored(torch, codes, scales, 64), perm.cpu().numpy(), k)
    np.testing.assert_array_equal(U.back(got), ref)
    n = int(off[-1])  # the rows that dispatch made, in 8 bits
    c2, s2 = qm.quantize_rows(rows, fmt, 64)
    assert torch.equal(got[:n], qm.dequantize_rows(c2, s2, x.dtype, 64)[:n])
    # entries outside the slots leave zeros, not reads
    bad = perm.clone()
    bad[0], bad[-1] = -1, T * k
    if T * k > 2:
        bad[1] = 2 ** 31 - 1
    got = qm.dequantize_rows(codes, scales, x.dtype, 64, perm=bad)
    np.testing.assert_array_equal(U.back(got), F.slots(V.stored(torch, codes, scales, 64), bad.cpu().numpy(), k))


def test_empty(torch):
    for shape in ((0, 8), (4, 0), (0, 0)):
        x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        c, s = qm.quantize_rows(x)
        assert c.shape == x.shape and s.shape == (shape[0], -(-shape[1] // 128))
        assert qm.dequantize_rows(c, s, torch.float16).shape == x.shape
    c, s = qm.quantize_rows(torch.zeros(0, 8, device="cuda"))
    assert qm.dequantize_rows(c, s, torch.float32, perm=torch.zeros(0, dtype=torch.int32, device="cuda")).shape == (0, 8)


def test_more_rows_than_one_launch_holds(torch):
    # a row a workgroup's thread of 16 columns: 2^22 workgroups of 1024 rows and more
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GiB of GPU memory")
    M = (1 << 26) + 3
    U.say(f"[rows8] {M} x 129")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-127, 128, (M, 129), generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    c, s = qm.quantize_rows(x, "int8", 128)
    for i in range(0, M, 1 << 23):  # every block's largest below 127.5: scales of 1 or less, values exact
        v = qm.dequantize_rows(c[i:i + (1 << 23)], s[i:i + (1 << 23)], torch.bfloat16)
        assert torch.equal(v, x[i:i + (1 << 23)]), i
    del v
    v = qm.dequantize_rows(c, s, torch.bfloat16)
    for i in range(0, M, 1 << 23):
        assert torch.equal(v[i:i + (1 << 23)], x[i:i + (1 << 23)]), i
