"""Refusals of the norm, routing from scores, rows in 8 bits and the linear
layers that leave and read them, on the host: every contract check runs before
anything is enqueued (pointers are never dereferenced by a refused call)."""
import ctypes
import os
import re

import numpy as np
import pytest

import quantized_mixture_experts_router_amd as qm

from test_steps_abi_cpu import GOOD, R, T, _a

NULL, SHAPE, ATTR, UNSUPPORTED, WORKSPACE, DTYPE, ALIGN = 1, 2, 3, 4, 5, 7, 8
F32, I32, I64, F16, BF16, F64, U8, E4 = qm.QMOE_F32, qm.QMOE_I32, qm.QMOE_I64, qm.QMOE_F16, qm.QMOE_BF16, qm.QMOE_F64, \
    qm.QMOE_U8, qm.QMOE_E4M3


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qm.LIB_PATH):
        pytest.skip("libqmoe.so not built (run __graft_entry__.build())")
    return qm.library()


def test_every_entry_point_of_the_header_is_exported_and_bound(lib):
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qmoe.h")).read()
    names = set(re.findall(r"\b(qmoe_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", src, flags=re.S)))
    assert {"qmoe_linear_q8", "qmoe_linear_backward_q8", "qmoe_rms_norm", "qmoe_route_scored"} <= names
    for n in names:
        assert hasattr(lib, n) and hasattr(qm, n), n


# ------------------------------------------------------------------ 8 bits
def _quantize(lib, x=T(BF16, 6, 40), block=16, c=T(U8, 6, 40), s=T(F32, 6, 3)):
    return lib.qmoe_quantize_rows(R(x), block, R(c), R(s), None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL), (dict(c=None), NULL), (dict(s=None), NULL), (dict(x=T(BF16, 6, 40, 1)), SHAPE),
    (dict(x=T(BF16, 240)), SHAPE), (dict(x=T(F64, 6, 40)), DTYPE), (dict(x=T(U8, 6, 40)), DTYPE),
    (dict(c=T(F16, 6, 40)), DTYPE), (dict(s=T(F16, 6, 3)), DTYPE), (dict(c=T(U8, 6, 41)), SHAPE),
    (dict(s=T(F32, 6, 2)), SHAPE), (dict(s=T(F32, 18)), SHAPE), (dict(x=T(BF16, -6, 40)), SHAPE),
    *[(dict(block=b), ATTR) for b in (0, -16, 8, 48, 256, 1 << 40)],
    (dict(x=T(BF16, (1 << 30) + 1, 1), c=T(U8, (1 << 30) + 1, 1), s=T(F32, (1 << 30) + 1, 1)), UNSUPPORTED),
    (dict(x=T(BF16, 1, 1 << 21), c=T(U8, 1, 1 << 21), s=T(F32, 1, 1 << 17)), UNSUPPORTED),
    (dict(x=T(BF16, 6, 40, ptr=None)), NULL), (dict(c=T(E4, 6, 40, ptr=None)), NULL),
    (dict(x=T(BF16, 6, 40, ptr=GOOD + 1)), ALIGN), (dict(s=T(F32, 6, 3, ptr=GOOD + 2)), ALIGN)])
def test_quantize_refusals(lib, kw, want):
    assert _quantize(lib, **kw) == want


def _dequantize(lib, c=T(E4, 6, 40), s=T(F32, 6, 3), block=16, p=None, o=T(F16, 6, 40)):
    return lib.qmoe_dequantize_rows(R(c), R(s), block, R(p), R(o), None)


@pytest.mark.parametrize("kw,want", [
    (dict(c=None), NULL), (dict(s=None), NULL), (dict(o=None), NULL), (dict(c=T(E4, 240)), SHAPE),
    (dict(c=T(F32, 6, 40)), DTYPE), (dict(s=T(I32, 6, 3)), DTYPE), (dict(o=T(F64, 6, 40)), DTYPE),
    (dict(o=T(U8, 6, 40)), DTYPE), (dict(o=T(F16, 6, 41)), SHAPE), (dict(o=T(F16, 5, 40)), SHAPE),
    (dict(s=T(F32, 6, 4)), SHAPE), (dict(block=17), ATTR), (dict(o=T(F16, -1, 40)), SHAPE),
    (dict(p=T(I64, 6)), DTYPE), (dict(p=T(I32, 6, 1)), SHAPE), (dict(p=T(I32, 12)), SHAPE),
    (dict(p=T(I32, 13), o=T(F16, 13, 40)), SHAPE),                     # not a whole number of slots a token
    (dict(c=T(E4, 0, 40), s=T(F32, 0, 3), p=T(I32, 4), o=T(F16, 4, 40)), SHAPE),
    (dict(c=T(E4, 6, 40, ptr=None)), NULL), (dict(p=T(I32, 12, ptr=GOOD + 2), o=T(F16, 12, 40)), ALIGN),
    (dict(c=T(E4, 1, 40), s=T(F32, 1, 3), p=T(I32, (1 << 30) + 1), o=T(F16, (1 << 30) + 1, 40)), UNSUPPORTED)])
def test_dequantize_refusals(lib, kw, want):
    assert _dequantize(lib, **kw) == want


# ------------------------------------------------------------------ norm
def _norm(lib, x=T(F16, 6, 40), r=T(F16, 6, 40), w=T(F16, 40), eps=1e-6, h=T(F16, 6, 40), y=T(F16, 6, 40), c=None, s=None,
          block=16):
    return lib.qmoe_rms_norm(R(x), R(r), R(w), eps, R(h), R(y), R(c), R(s), block, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL), (dict(y=None), NULL), (dict(r=None), NULL),  # a sum without a residual
    (dict(c=T(U8, 6, 40)), NULL), (dict(s=T(F32, 6, 3)), NULL), (dict(x=T(F16, 6, 40, 1)), SHAPE),
    (dict(r=T(F16, 6)), SHAPE), (dict(w=T(F16, 1, 40)), SHAPE), (dict(w=T(F16, 41)), SHAPE), (dict(y=T(F16, 6, 39)), SHAPE),
    (dict(h=T(F16, 5, 40)), SHAPE), (dict(r=T(F16, 1, 40)), SHAPE), (dict(x=T(F64, 6, 40)), DTYPE), (dict(r=T(F32, 6, 40)), DTYPE),
    (dict(w=T(F32, 40)), DTYPE), (dict(y=T(BF16, 6, 40)), DTYPE), (dict(h=T(F32, 6, 40)), DTYPE),
    *[(dict(eps=e), ATTR) for e in (0.0, -1e-6, float("nan"), float("inf"))],
    (dict(c=T(F16, 6, 40), s=T(F32, 6, 3)), DTYPE), (dict(c=T(U8, 6, 40), s=T(F32, 6, 3), block=24), ATTR),
    (dict(c=T(U8, 6, 40), s=T(F32, 6, 2)), SHAPE), (dict(x=T(F16, 6, 40, ptr=None)), NULL),
    (dict(w=T(F16, 40, ptr=GOOD + 1)), ALIGN), (dict(y=T(F16, 6, 40, ptr=None)), NULL),
    (dict(x=T(F16, 1, 1 << 21), r=None, w=None, h=None, y=T(F16, 1, 1 << 21)), UNSUPPORTED)])
def test_norm_refusals(lib, kw, want):
    assert _norm(lib, **kw) == want


def _norm_back(lib, g=T(F32, 6, 40), ds=T(F32, 6, 40), x=T(F32, 6, 40), w=T(F32, 40), eps=1e-6, gi=T(F32, 6, 40),
               gw=T(F32, 40), ws=GOOD, n=1 << 20):
    return lib.qmoe_rms_norm_backward(R(g), R(ds), R(x), R(w), eps, R(gi), R(gw), ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(g=None), NULL), (dict(x=None), NULL), (dict(w=None), NULL), (dict(g=T(F16, 6, 40)), DTYPE),
    (dict(ds=T(F16, 6, 40)), DTYPE), (dict(gi=T(F16, 6, 40)), DTYPE), (dict(gw=T(F16, 40)), DTYPE), (dict(w=T(F16, 40)), DTYPE),
    (dict(ds=T(F32, 6, 41)), SHAPE), (dict(gi=T(F32, 7, 40)), SHAPE), (dict(gw=T(F32, 39)), SHAPE), (dict(gw=T(F32, 1, 40)), SHAPE),
    (dict(eps=0.0), ATTR), (dict(ws=None), NULL), (dict(n=40 * 4 - 1), WORKSPACE), (dict(ws=GOOD + 16), ALIGN),
    (dict(gi=T(F32, 6, 40, ptr=None)), NULL), (dict(g=T(F32, 6, 40, ptr=GOOD + 2)), ALIGN)])
def test_norm_backward_refusals(lib, kw, want):
    assert _norm_back(lib, **kw) == want


def test_norm_workspace(lib):
    x, w = np.zeros((3, 10), np.float16), np.zeros(10, np.float16)
    size = lambda x, w, gw: qm.qmoe_rms_norm_backward_workspace_size(x, None, x, w, 1e-6, x, gw)  # noqa: E731
    assert size(x, w, None) == 0 and size(x[:0], w, w) == 0
    assert size(x, w, w) == 12 * 4  # one row of sums of a workgroup's rows, whole fours of columns
    assert size(np.broadcast_to(x[:1], (33, 10)), w, w) == 2 * 12 * 4
    big = np.broadcast_to(x[:1, :1], (1 << 20, 4096))
    assert 0 < size(big, np.broadcast_to(w[:1], (4096,)), np.broadcast_to(w[:1], (4096,))) <= 1 << 25


# ------------------------------------------------------------------ routing from scores
def _attrs(**kw):
    a = qm.qmoe_route_attrs_default()
    for k, v in dict(dict(k=2), **kw).items():
        setattr(a, k, v)
    return a


def test_route_attrs(lib):
    a, b = qm.qmoe_route_attrs_default(), qm.make_route_attrs()
    assert bytes(a) == bytes(b)
    assert (a.k, a.scores, a.groups, a.kept_groups, a.group_top, a.normalize_routing_weights, a.scale) == (1, 0, 1, 1, 2, 0, 1)
    with pytest.raises(ValueError):
        qm.make_route_attrs({"routing": "moe"})


def _route(lib, l=T(F32, 5, 8), b=T(F32, 8), a={}, i=T(I32, 5, 2), w=T(F32, 5, 2)):
    return lib.qmoe_route_scored(R(l), R(b), R(_attrs(**a)) if a is not None else None, R(i), R(w), None)


BAD_ATTRS = [dict(scores=2), dict(scores=-1), dict(groups=0), dict(groups=3), dict(groups=-2), dict(groups=16),
             dict(groups=4, kept_groups=5), dict(groups=4, kept_groups=0), dict(group_top=0), dict(group_top=3),
             dict(normalize_routing_weights=2), dict(scale=float("nan")), dict(scale=float("inf"))]


@pytest.mark.parametrize("kw,want", [
    (dict(l=None), NULL), (dict(a=None), NULL), (dict(i=None), NULL), (dict(w=None), NULL), (dict(l=T(F16, 5, 8)), DTYPE),
    (dict(l=T(F32, 5, 8, 1)), SHAPE), (dict(l=T(F32, -5, 8)), SHAPE), (dict(b=T(F32, 7)), SHAPE), (dict(b=T(F32, 1, 8)), SHAPE),
    (dict(b=T(F16, 8)), DTYPE), (dict(i=T(I64, 5, 2)), DTYPE), (dict(w=T(F16, 5, 2)), DTYPE), (dict(i=T(I32, 5, 3)), SHAPE),
    (dict(w=T(F32, 10)), SHAPE), *[(dict(a=a), ATTR) for a in BAD_ATTRS + [dict(k=0), dict(k=9), dict(k=3, groups=4, kept_groups=1)]],
    (dict(l=T(F32, 5, 1025), b=None), UNSUPPORTED), (dict(l=T(F32, 5, 130), b=None, a=dict(groups=65)), UNSUPPORTED),
    (dict(l=T(F32, 1 << 29, 8)), UNSUPPORTED), (dict(l=T(F32, 5, 8, ptr=None)), NULL),
    (dict(b=T(F32, 8, ptr=GOOD + 2)), ALIGN), (dict(w=T(F32, 5, 2, ptr=None)), NULL)])
def test_route_refusals(lib, kw, want):
    assert _route(lib, **kw) == want


def _route_back(lib, g=T(F32, 5, 2), l=T(F32, 5, 8), i=T(I64, 5, 2), a={}, o=T(F32, 5, 8)):
    return lib.qmoe_route_scored_backward(R(g), R(l), R(i), R(_attrs(**a)) if a is not None else None, R(o), None)


@pytest.mark.parametrize("kw,want", [
    (dict(g=None), NULL), (dict(l=None), NULL), (dict(i=None), NULL), (dict(a=None), NULL), (dict(o=None), NULL),
    (dict(i=T(I32, 5)), SHAPE), (dict(i=T(I32, 5, 0)), ATTR), (dict(i=T(I32, 5, 9)), ATTR), (dict(i=T(F32, 5, 2)), DTYPE),
    (dict(g=T(F32, 5, 3)), SHAPE), (dict(o=T(F32, 5, 7)), SHAPE), (dict(g=T(F16, 5, 2)), DTYPE),
    *[(dict(a=a), ATTR) for a in BAD_ATTRS], (dict(i=T(I64, 5, 2, ptr=GOOD + 4)), ALIGN)])
def test_route_backward_refusals(lib, kw, want):
    assert _route_back(lib, **kw) == want


# ------------------------------------------------------------------ linear layers
def _linear(lib, x=T(BF16, 6, 16), w=T(BF16, 40, 16), b=T(BF16, 40), r=T(BF16, 6, 40), off=None, a={}, y=T(BF16, 6, 40),
            c=T(U8, 6, 40), s=T(F32, 6, 3), block=16, ws=None, n=0):
    return lib.qmoe_linear_q8(R(x), R(w), R(b), R(r), R(off), R(_a(**a)) if a is not None else None, R(y), R(c), R(s),
                              block, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(a=None), NULL), (dict(y=None), NULL), (dict(c=None), NULL),
    (dict(s=None), NULL), (dict(c=T(BF16, 6, 40)), DTYPE), (dict(s=T(BF16, 6, 3)), DTYPE), (dict(c=T(E4, 6, 39)), SHAPE),
    (dict(s=T(F32, 6, 4)), SHAPE), (dict(block=0), ATTR), (dict(w=T(F16, 40, 16)), DTYPE), (dict(x=T(U8, 6, 16)), DTYPE),
    (dict(a=dict(activation_type=7)), ATTR), (dict(c=T(U8, 6, 40, ptr=None)), NULL), (dict(s=T(F32, 6, 3, ptr=GOOD + 1)), ALIGN),
    (dict(x=T(BF16, 6, 16, ptr=GOOD + 2)), ALIGN), (dict(x=T(BF16, 6, 15), w=T(BF16, 40, 15)), NULL),
    (dict(x=T(BF16, 6, 15), w=T(BF16, 40, 15), ws=GOOD, n=16), WORKSPACE)])
def test_linear_q8_refusals(lib, kw, want):
    assert _linear(lib, **kw) == want


SILU = dict(activation_type=qm.QMOE_ACT["silu"])


def _back(lib, g=T(F16, 6, 8), x=T(U8, 6, 16), xs=T(F32, 6, 1), p=None, w=T(F16, 8, 16), z=T(E4, 6, 8), zs=T(F32, 6, 1),
          block=16, off=None, a=SILU, gi=T(F16, 6, 16), gw=T(F16, 8, 16), gb=T(F16, 8), ws=GOOD, n=1 << 20):
    return lib.qmoe_linear_backward_q8(R(g), R(x), R(xs), R(p), R(w), R(z), R(zs), block, R(off),
                                       R(_a(**a)) if a is not None else None, R(gi), R(gw), R(gb), ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(g=None), NULL), (dict(x=None), NULL), (dict(w=None), NULL), (dict(a=None), NULL), (dict(xs=None), NULL),
    (dict(zs=None), NULL), (dict(z=None, zs=None), NULL), (dict(z=None), DTYPE),
    (dict(x=T(F16, 6, 16)), DTYPE), (dict(z=T(F16, 6, 8)), DTYPE),     # scales beside what is not in 8 bits
    (dict(x=T(F16, 6, 16), xs=None, p=T(I32, 6)), DTYPE),              # perm beside it
    (dict(x=T(F32, 6, 16), xs=None), DTYPE), (dict(z=T(F32, 6, 8), zs=None), DTYPE), (dict(w=T(U8, 8, 16)), DTYPE),
    (dict(xs=T(F16, 6, 1)), DTYPE), (dict(zs=T(I32, 6, 1)), DTYPE), (dict(xs=T(F32, 6, 2)), SHAPE), (dict(zs=T(F32, 5, 1)), SHAPE),
    (dict(x=T(U8, 5, 16), xs=T(F32, 5, 1)), SHAPE), (dict(z=T(E4, 6, 9)), SHAPE), (dict(z=T(E4, 48)), SHAPE),
    (dict(p=T(I64, 6)), DTYPE), (dict(p=T(I32, 6, 1)), SHAPE), (dict(p=T(I32, 12)), SHAPE),
    (dict(p=T(I32, 6), x=T(U8, 4, 16), xs=T(F32, 4, 1)), SHAPE), (dict(p=T(I32, 6), x=T(U8, 0, 16), xs=T(F32, 0, 1)), SHAPE),
    (dict(block=20), ATTR), (dict(g=T(F32, 6, 8)), DTYPE), (dict(gi=T(F16, 6, 15)), SHAPE), (dict(gb=T(F16, 9)), SHAPE),
    (dict(ws=None), NULL), (dict(n=4), WORKSPACE), (dict(ws=GOOD + 4), ALIGN), (dict(x=T(U8, 6, 16, ptr=None)), NULL),
    (dict(xs=T(F32, 6, 1, ptr=GOOD + 2)), ALIGN), (dict(p=T(I32, 6, ptr=GOOD + 2)), ALIGN)])
def test_linear_backward_q8_refusals(lib, kw, want):
    assert _back(lib, **kw) == want


def test_linear_q8_workspaces(lib):
    x, w = np.zeros((4, 16), np.float16), np.zeros((8, 16), np.float16)
    c, s = np.zeros((4, 8), np.uint8), np.zeros((4, 1), np.float32)
    assert qm.qmoe_linear_q8_workspace_size(x, w, codes=c, scales=s) == qm.qmoe_linear_workspace_size(x, w) == 0
    x8, xs = np.zeros((2, 16), np.uint8), np.zeros((2, 1), np.float32)
    size = lambda gw: qm.qmoe_linear_backward_q8_workspace_size(  # noqa: E731
        np.zeros((4, 8), np.float16), (x8, xs), w, (c, s), None, {"activation_type": "relu"}, x, gw, None, 128,
        np.zeros(4, np.int32))
    assert size(None) == 256                # the gradient of the activation
    assert size(w) == 256 + 256             # and the input's rows
    with pytest.raises(qm.QmoeError) as e:
        qm.qmoe_linear_q8_workspace_size(x, w, codes=c, scales=s, block_size=12)
    assert e.value.name == "ATTR"


def test_python_refuses_other_formats_and_devices(lib):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        qm.rms_norm(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        qm.quantize_rows(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        qm._code_type("e5m2")
    assert ctypes.sizeof(qm.QmoeRouteAttrs) == 28
