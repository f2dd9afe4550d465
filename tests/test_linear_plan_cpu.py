"""The plan of the linear layers' products (host code): its refusals, and that
the shapes of the GPU tests reach every kind of product."""
import ctypes
import os

import pytest

import quantized_mixture_experts_router_amd as qm

import linear_shapes as L

NULL, SHAPE, UNSUPPORTED, DTYPE = 1, 2, 4, 7


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qm.LIB_PATH):
        pytest.skip("libqmoe.so not built (run __graft_entry__.build())")
    return qm.library()


def T(dtype, *dims):
    t = qm.QmoeTensor()
    t.data, t.dtype, t.rank = None, dtype, len(dims)
    for i, d in enumerate(dims[:3]):
        t.dims[i] = d
    return t


def plan(lib, dt, M, K, N, G=0, off=True):
    buf = ctypes.create_string_buffer(128)
    code = qm.QMOE_F32 if dt == "float32" else qm.QMOE_BF16
    x, w = T(code, M, K), T(code, G, N, K) if G else T(code, N, K)
    o = ctypes.byref(T(qm.QMOE_I32, G + 1)) if G and off else None
    st = lib.qmoe_linear_plan_describe(ctypes.byref(x), ctypes.byref(w), o, buf, 128)
    return st, buf.value.decode()


@pytest.mark.parametrize("dt", sorted(L.SHAPES))
def test_shapes_reach_every_kind_of_product(lib, dt):
    seen = set()
    for s in L.SHAPES[dt]:
        st, text = plan(lib, dt, *s)
        assert st == 0
        seen |= L.kinds(text, dt, *s)
    missing = L.all_kinds(dt) - seen
    assert not missing, sorted(missing)
    assert not seen - L.all_kinds(dt), sorted(seen - L.all_kinds(dt))


def test_plan_text_and_refusals(lib):
    assert plan(lib, "16bit", 3000, 3336, 4104) == (0, "forward=256x256:1 grad_input=256x256:1 grad_weights=256x256:1")
    assert plan(lib, "16bit", 0, 16, 16)[0] == 0
    assert plan(lib, "16bit", 8, 16, 16, 3, off=False)[0] == NULL
    assert plan(lib, "16bit", 8, 1 << 21, 16)[0] == UNSUPPORTED
    assert plan(lib, "16bit", -1, 16, 16)[0] == SHAPE
    x = T(qm.QMOE_F64, 4, 4)
    buf = ctypes.create_string_buffer(8)
    f = lib.qmoe_linear_plan_describe
    assert f(ctypes.byref(x), ctypes.byref(x), None, buf, 8) == DTYPE
    y = T(qm.QMOE_F32, 4, 4)
    assert f(ctypes.byref(y), ctypes.byref(y), None, None, 8) == NULL
    assert f(ctypes.byref(y), ctypes.byref(y), None, buf, 0) == NULL
    assert f(None, ctypes.byref(y), None, buf, 8) == NULL
    assert f(ctypes.byref(y), ctypes.byref(y), None, buf, 8) == 0 and buf.value == b"forward"  # cut to the buffer
