"""Python binding of libqmoe.so, the QMoE routed expert FFN for gfx950.

Argument marshalling only: every step of the operator runs in the HIP
kernels behind the C ABI of include/qmoe.h.  PyTorch supplies device memory
and the current stream.  The functions keep the C names:

    qmoe_abi_version, qmoe_attrs_default, qmoe_validate, qmoe_workspace_size,
    qmoe_plan_describe, qmoe_forward, qmoe_forward_debug, qmoe_forward_noalloc,
    qmoe_noalloc_scratch_bytes, qmoe_status_string,
    qmoe_grouped_matmul_workspace_size, qmoe_grouped_matmul,
    qmoe_grouped_matmul_debug, qmoe_moe_attrs_default, qmoe_moe_validate,
    qmoe_moe_workspace_size, qmoe_moe_forward, qmoe_moe_forward_debug,
    qmoe_route, qmoe_route_backward, qmoe_dispatch_workspace_size,
    qmoe_dispatch, qmoe_dispatch_backward, qmoe_combine,
    qmoe_combine_backward, qmoe_linear_attrs_default,
    qmoe_linear_plan_describe, qmoe_linear_workspace_size, qmoe_linear,
    qmoe_linear_backward_workspace_size, qmoe_linear_backward,
    qmoe_quantize_rows, qmoe_dequantize_rows, qmoe_rms_norm,
    qmoe_rms_norm_backward_workspace_size, qmoe_rms_norm_backward,
    qmoe_route_attrs_default, qmoe_route_scored, qmoe_route_scored_backward,
    qmoe_linear_q8_workspace_size, qmoe_linear_q8,
    qmoe_linear_backward_q8_workspace_size, qmoe_linear_backward_q8

plus ``forward``, ``grouped_matmul`` and ``moe_forward`` (allocate output and
workspace with torch, then call the entry point) for convenience, and the
same for the steps of a routed layer and their gradients: ``route``,
``dispatch``, ``combine``, ``linear`` and their ``*_backward``, and for what
stands around them: ``rms_norm``, ``route_scored``, ``quantize_rows``,
``dequantize_rows``, ``linear_q8``, ``linear_backward_q8``.  The
library is loaded on first use; a missing build raises immediately, there is
no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import struct
import threading
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqmoe.so")

QMOE_F32, QMOE_U8, QMOE_I32, QMOE_I64, QMOE_F16, QMOE_BF16, QMOE_F64, QMOE_E4M3 = 1, 2, 3, 4, 5, 6, 7, 8
QMOE_ACT = {"relu": 0, "swiglu": 1, "gelu": 2, "silu": 3, "identity": 4}
QMOE_ROUTING = {"qmoe": 0, "moe": 1}
QMOE_SCORES = {"softmax": 0, "sigmoid": 1}
STATUS = {0: "OK", 1: "NULL", 2: "SHAPE", 3: "ATTR", 4: "UNSUPPORTED", 5: "WORKSPACE", 6: "HIP",
          7: "DTYPE", 8: "ALIGN"}


class QmoeTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("dims", ctypes.c_int64 * 3)]


class QmoeAttrs(ctypes.Structure):
    _fields_ = [("k", ctypes.c_int32), ("expert_weight_bits", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("activation_type", ctypes.c_int32), ("swiglu_fusion", ctypes.c_int32),
                ("activation_alpha", ctypes.c_float), ("activation_beta", ctypes.c_float),
                ("normalize_routing_weights", ctypes.c_int32), ("routing", ctypes.c_int32),
                ("use_sparse_mixer", ctypes.c_int32), ("weights_prepacked", ctypes.c_int32),
                ("quant_type", ctypes.c_int32), ("has_swiglu_limit", ctypes.c_int32),
                ("swiglu_limit", ctypes.c_float), ("first_expert", ctypes.c_int32)]


class QmoeMoeAttrs(ctypes.Structure):
    _fields_ = [("k", ctypes.c_int32), ("activation_type", ctypes.c_int32), ("swiglu_fusion", ctypes.c_int32),
                ("activation_alpha", ctypes.c_float), ("activation_beta", ctypes.c_float),
                ("normalize_routing_weights", ctypes.c_int32), ("use_sparse_mixer", ctypes.c_int32),
                ("has_swiglu_limit", ctypes.c_int32), ("swiglu_limit", ctypes.c_float)]


class QmoeLinearAttrs(ctypes.Structure):
    _fields_ = [("activation_type", ctypes.c_int32), ("swiglu_fusion", ctypes.c_int32),
                ("activation_alpha", ctypes.c_float), ("activation_beta", ctypes.c_float),
                ("has_swiglu_limit", ctypes.c_int32), ("swiglu_limit", ctypes.c_float)]


class QmoeRouteAttrs(ctypes.Structure):
    _fields_ = [("k", ctypes.c_int32), ("scores", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("kept_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("normalize_routing_weights", ctypes.c_int32), ("scale", ctypes.c_float)]


QMOE_STAGE_EVENTS = 6
QMOE_GMM_EVENTS = 3


class QmoeDebug(ctypes.Structure):
    _fields_ = [("topk_idx", ctypes.c_void_p), ("topk_w", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("perm", ctypes.c_void_p),
                ("events", ctypes.c_void_p * QMOE_STAGE_EVENTS)]


class QmoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS.get(status, status)} ({qmoe_status_string(status)})")
        self.status = status
        self.name = STATUS.get(status, str(status))


_lib_handle = None


def _lib():
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m quantized_mixture_experts_router_amd.build`")
        # torch ships its own HIP runtime under the same soname; loading torch
        # first makes this library bind to that one copy (one runtime per process).
        import torch  # noqa: F401
        lib = ctypes.CDLL(LIB_PATH)
        T = ctypes.POINTER(QmoeTensor)
        A = ctypes.POINTER(QmoeAttrs)
        lib.qmoe_abi_version.restype = ctypes.c_int32
        lib.qmoe_attrs_default.argtypes = [A]
        lib.qmoe_attrs_default.restype = None
        lib.qmoe_validate.argtypes = [T, T, T, T, T, T, T, A]
        lib.qmoe_validate.restype = ctypes.c_int
        lib.qmoe_workspace_size.argtypes = [T, T, T, T, T, T, A, ctypes.POINTER(ctypes.c_size_t)]
        lib.qmoe_workspace_size.restype = ctypes.c_int
        lib.qmoe_forward.argtypes = [T, T, T, T, T, T, A, T, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.qmoe_forward.restype = ctypes.c_int
        lib.qmoe_forward_debug.argtypes = [T, T, T, T, T, T, A, T, ctypes.c_void_p, ctypes.c_size_t,
                                           ctypes.c_void_p, ctypes.POINTER(QmoeDebug)]
        lib.qmoe_forward_debug.restype = ctypes.c_int
        lib.qmoe_plan_describe.argtypes = [T, T, T, T, T, T, A, ctypes.c_char_p, ctypes.c_size_t]
        lib.qmoe_plan_describe.restype = ctypes.c_int
        lib.qmoe_noalloc_scratch_bytes.argtypes = []
        lib.qmoe_noalloc_scratch_bytes.restype = ctypes.c_size_t
        lib.qmoe_forward_noalloc.argtypes = [T, T, T, T, T, T, A, T, ctypes.c_void_p]
        lib.qmoe_forward_noalloc.restype = ctypes.c_int
        lib.qmoe_grouped_matmul_workspace_size.argtypes = [T, T, T, T, T, ctypes.POINTER(ctypes.c_size_t)]
        lib.qmoe_grouped_matmul_workspace_size.restype = ctypes.c_int
        lib.qmoe_grouped_matmul.argtypes = [T, T, T, T, T, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.qmoe_grouped_matmul.restype = ctypes.c_int
        lib.qmoe_grouped_matmul_debug.argtypes = [T, T, T, T, T, ctypes.c_void_p, ctypes.c_size_t,
                                                  ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)]
        lib.qmoe_grouped_matmul_debug.restype = ctypes.c_int
        MA = ctypes.POINTER(QmoeMoeAttrs)
        lib.qmoe_moe_attrs_default.argtypes = [MA]
        lib.qmoe_moe_attrs_default.restype = None
        lib.qmoe_moe_validate.argtypes = [T] * 9 + [MA]
        lib.qmoe_moe_validate.restype = ctypes.c_int
        lib.qmoe_moe_workspace_size.argtypes = [T] * 8 + [MA, ctypes.POINTER(ctypes.c_size_t)]
        lib.qmoe_moe_workspace_size.restype = ctypes.c_int
        lib.qmoe_moe_forward.argtypes = [T] * 8 + [MA, T, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.qmoe_moe_forward.restype = ctypes.c_int
        lib.qmoe_moe_forward_debug.argtypes = [T] * 8 + [MA, T, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                                         ctypes.POINTER(QmoeDebug)]
        lib.qmoe_moe_forward_debug.restype = ctypes.c_int
        LA, I32, I64, P, Z = (ctypes.POINTER(QmoeLinearAttrs), ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p,
                              ctypes.c_size_t)
        ZP, RA, F = ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(QmoeRouteAttrs), ctypes.c_float
        D = P  # tensors as addresses into the packed arguments (_pack)
        for name, args in (("qmoe_route", [D, I32, I32, I32, D, D, P]),
                           ("qmoe_route_backward", [D, D, D, I32, I32, D, P]),
                           ("qmoe_dispatch_workspace_size", [D, D, I64, ZP]),
                           ("qmoe_dispatch", [D, D, I64, D, D, D, D, P, Z, P]),
                           ("qmoe_dispatch_backward", [D, D, D, P]),
                           ("qmoe_combine", [D, D, D, D, P]),
                           ("qmoe_combine_backward", [D] * 6 + [P]),
                           ("qmoe_linear_plan_describe", [D, D, D, ctypes.c_char_p, Z]),
                           ("qmoe_linear_workspace_size", [D] * 5 + [LA, D, D, ZP]),
                           ("qmoe_linear", [D] * 5 + [LA, D, D, P, Z, P]),
                           ("qmoe_linear_backward_workspace_size", [D] * 5 + [LA, D, D, D, ZP]),
                           ("qmoe_linear_backward", [D] * 5 + [LA, D, D, D, P, Z, P]),
                           ("qmoe_quantize_rows", [D, I64, D, D, P]),
                           ("qmoe_dequantize_rows", [D, D, I64, D, D, P]),
                           ("qmoe_rms_norm", [D, D, D, F, D, D, D, D, I64, P]),
                           ("qmoe_rms_norm_backward_workspace_size", [D, D, D, D, F, D, D, ZP]),
                           ("qmoe_rms_norm_backward", [D, D, D, D, F, D, D, P, Z, P]),
                           ("qmoe_route_scored", [D, D, RA, D, D, P]),
                           ("qmoe_route_scored_backward", [D, D, D, RA, D, P]),
                           ("qmoe_linear_q8_workspace_size", [D] * 5 + [LA, D, D, D, I64, ZP]),
                           ("qmoe_linear_q8", [D] * 5 + [LA, D, D, D, I64, P, Z, P]),
                           ("qmoe_linear_backward_q8_workspace_size", [D] * 7 + [I64, D, LA, D, D, D, ZP]),
                           ("qmoe_linear_backward_q8", [D] * 7 + [I64, D, LA, D, D, D, P, Z, P])):
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = ctypes.c_int
        lib.qmoe_linear_attrs_default.argtypes = [LA]
        lib.qmoe_linear_attrs_default.restype = None
        lib.qmoe_route_attrs_default.argtypes = [RA]
        lib.qmoe_route_attrs_default.restype = None
        lib.qmoe_status_string.argtypes = [ctypes.c_int]
        lib.qmoe_status_string.restype = ctypes.c_char_p
        _lib_handle = lib
    return _lib_handle


def library():
    """The loaded ctypes library (raises if it is not built)."""
    return _lib()


# ------------------------------------------------------------------ marshalling
def describe(t, data: bool = True) -> QmoeTensor:
    """qmoe_tensor for a torch tensor or numpy array (shape, dtype, pointer)."""
    shape = tuple(t.shape)  # ranks above 3 pass through so the library rejects them
    name = str(t.dtype).replace("torch.", "")
    code = {"float32": QMOE_F32, "uint8": QMOE_U8, "int32": QMOE_I32, "int64": QMOE_I64, "float16": QMOE_F16,
            "bfloat16": QMOE_BF16, "float64": QMOE_F64, "float8_e4m3fn": QMOE_E4M3}.get(name, 0)
    ptr = None
    if data and hasattr(t, "data_ptr"):
        if not t.is_contiguous():
            raise ValueError("qmoe tensors must be contiguous")
        ptr = t.data_ptr() if t.numel() > 0 else None
    d = QmoeTensor()
    d.data = ptr
    d.dtype = code
    d.rank = len(shape)
    for i in range(3):
        d.dims[i] = shape[i] if i < len(shape) else 0
    return d


def make_attrs(attrs: Optional[dict] = None) -> QmoeAttrs:
    a = qmoe_attrs_default()
    for key, val in (attrs or {}).items():
        if key == "activation_type":
            val = QMOE_ACT.get(val, 99) if isinstance(val, str) else val
        elif key == "routing":
            val = QMOE_ROUTING.get(val, 99) if isinstance(val, str) else val
        elif key == "quant_type":
            val = 0 if val in ("int", 0) else 1
        elif key == "block_size" and val is None:
            val = 0
        elif key == "swiglu_limit":
            # absent (None) or a value; a given value is passed as is and
            # the library checks it
            a.has_swiglu_limit = 0 if val is None else 1
            val = 0.0 if val is None else val
        setattr(a, key, val)
    return a


# ------------------------------------------------------------------ C entry points
def qmoe_abi_version() -> int:
    return int(_lib().qmoe_abi_version())


def qmoe_status_string(status: int) -> str:
    return _lib().qmoe_status_string(int(status)).decode()


def qmoe_attrs_default() -> QmoeAttrs:
    a = QmoeAttrs()
    _lib().qmoe_attrs_default(ctypes.byref(a))
    return a


def _six(input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s, data=True):
    return [describe(t, data) for t in (input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s)]


def qmoe_validate(input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s, output=None, attrs=None) -> int:
    """Status code of the contract check (0 = OK).  Arrays may live anywhere."""
    ts = _six(input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s, data=False)
    out = ctypes.byref(describe(output, False)) if output is not None else None
    a = attrs if isinstance(attrs, QmoeAttrs) else make_attrs(attrs)
    return int(_lib().qmoe_validate(*[ctypes.byref(t) for t in ts], out, ctypes.byref(a)))


def qmoe_workspace_size(input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s, attrs=None) -> int:
    ts = _six(input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s, data=False)
    a = attrs if isinstance(attrs, QmoeAttrs) else make_attrs(attrs)
    n = ctypes.c_size_t(0)
    st = _lib().qmoe_workspace_size(*[ctypes.byref(t) for t in ts], ctypes.byref(a), ctypes.byref(n))
    if st != 0:
        raise QmoeError(st, "qmoe_workspace_size")
    return int(n.value)


def qmoe_plan_describe(input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s, attrs=None) -> str:
    """The launch plan of qmoe_forward for these shapes, as one line of text.
    Arrays may live anywhere (only shapes and dtypes are read)."""
    ts = _six(input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s, data=False)
    a = attrs if isinstance(attrs, QmoeAttrs) else make_attrs(attrs)
    buf = ctypes.create_string_buffer(512)
    st = _lib().qmoe_plan_describe(*[ctypes.byref(t) for t in ts], ctypes.byref(a), buf, 512)
    if st != 0:
        raise QmoeError(st, "qmoe_plan_describe")
    return buf.value.decode()


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def qmoe_forward(input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s, attrs, output, workspace, stream=None,
                 debug: Optional[dict] = None) -> None:
    """Enqueue the operator on ``stream`` (default: torch's current stream).

    All tensors are contiguous device tensors; ``workspace`` is a uint8 device
    tensor of at least qmoe_workspace_size bytes (or None when that size is 0).
    ``debug`` may map topk_idx / topk_w / counts / offsets / perm to device
    tensors that receive the routing stages' results, and ``events`` to up to
    QMOE_STAGE_EVENTS raw hipEvent_t handles (qmoe_forward_debug).
    """
    ts = _six(input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s)
    o = describe(output)
    a = attrs if isinstance(attrs, QmoeAttrs) else make_attrs(attrs)
    wptr = workspace.data_ptr() if workspace is not None and workspace.numel() > 0 else None
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = [*[ctypes.byref(t) for t in ts], ctypes.byref(a), ctypes.byref(o), ctypes.c_void_p(wptr),
            ctypes.c_size_t(wbytes), _stream_handle(stream)]
    if debug is None:
        st = _lib().qmoe_forward(*args)
        where = "qmoe_forward"
    else:
        dbg = QmoeDebug()
        for f in ("topk_idx", "topk_w", "counts", "offsets", "perm"):
            t = debug.get(f)
            setattr(dbg, f, t.data_ptr() if t is not None and t.numel() > 0 else None)
        for i, ev in enumerate(debug.get("events") or ()):
            dbg.events[i] = ev  # raw hipEvent_t handles
        st = _lib().qmoe_forward_debug(*args, ctypes.byref(dbg))
        where = "qmoe_forward_debug"
    if st != 0:
        raise QmoeError(st, where)


qmoe_forward_debug = qmoe_forward


def qmoe_noalloc_scratch_bytes() -> int:
    """Size of the library's per-GPU scratch array used by qmoe_forward_noalloc."""
    return int(_lib().qmoe_noalloc_scratch_bytes())


def qmoe_forward_noalloc(input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s, attrs, output, stream=None) -> None:
    """qmoe_forward without a workspace: the library's per-GPU scratch array
    holds the intermediates (calls on one GPU must not overlap)."""
    ts = _six(input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s)
    o = describe(output)
    a = attrs if isinstance(attrs, QmoeAttrs) else make_attrs(attrs)
    st = _lib().qmoe_forward_noalloc(*[ctypes.byref(t) for t in ts], ctypes.byref(a), ctypes.byref(o),
                                     _stream_handle(stream))
    if st != 0:
        raise QmoeError(st, "qmoe_forward_noalloc")


def forward(input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s, attrs=None, stream=None, workspace=None,
            output=None, debug=None):
    """Allocate output (and workspace unless given) with torch, then qmoe_forward."""
    import torch
    if output is None:
        output = torch.empty_like(input)
    need = qmoe_workspace_size(input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s, attrs)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=input.device)
    qmoe_forward(input, router_probs, fc1_w, fc1_s, fc2_w, fc2_s, attrs, output, workspace, stream, debug)
    return output


def _ref(t, data):
    return ctypes.byref(describe(t, data)) if t is not None else None


def qmoe_grouped_matmul_workspace_size(input, weights, group_indices, bias=None, output=None) -> int:
    """Workspace bytes of qmoe_grouped_matmul.  Arrays may live anywhere."""
    n = ctypes.c_size_t(0)
    st = _lib().qmoe_grouped_matmul_workspace_size(_ref(input, False), _ref(weights, False),
                                                   _ref(group_indices, False), _ref(bias, False),
                                                   _ref(output, False), ctypes.byref(n))
    if st != 0:
        raise QmoeError(st, "qmoe_grouped_matmul_workspace_size")
    return int(n.value)


def qmoe_grouped_matmul(input, weights, group_indices, bias, output, workspace, stream=None, events=None) -> None:
    """Enqueue GroupedMatMul on ``stream`` (default: torch's current stream).

    Contiguous device tensors; ``bias`` may be None; ``workspace`` a uint8
    device tensor of at least qmoe_grouped_matmul_workspace_size bytes (or
    None when that size is 0).  ``events``: up to QMOE_GMM_EVENTS raw
    hipEvent_t handles (calls qmoe_grouped_matmul_debug).
    """
    wptr = workspace.data_ptr() if workspace is not None and workspace.numel() > 0 else None
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = [_ref(input, True), _ref(weights, True), _ref(group_indices, True), _ref(bias, True),
            _ref(output, True), ctypes.c_void_p(wptr), ctypes.c_size_t(wbytes), _stream_handle(stream)]
    if events is None:
        st = _lib().qmoe_grouped_matmul(*args)
        where = "qmoe_grouped_matmul"
    else:
        ev = (ctypes.c_void_p * QMOE_GMM_EVENTS)()
        for i, e in enumerate(events):
            ev[i] = e
        st = _lib().qmoe_grouped_matmul_debug(*args, ev)
        where = "qmoe_grouped_matmul_debug"
    if st != 0:
        raise QmoeError(st, where)


def grouped_matmul(input, weights, group_indices, bias=None, stream=None, workspace=None, output=None):
    """Allocate output [M, S, N] (and workspace unless given) with torch, then qmoe_grouped_matmul."""
    import torch
    if output is None:
        output = torch.empty((input.shape[0], group_indices.shape[1], weights.shape[2]), dtype=input.dtype,
                             device=input.device)
    need = qmoe_grouped_matmul_workspace_size(input, weights, group_indices, bias, output)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=input.device)
    qmoe_grouped_matmul(input, weights, group_indices, bias, output, workspace, stream)
    return output


qmoe_grouped_matmul_debug = qmoe_grouped_matmul


# ------------------------------------------------------------------ float MoE
MOE_TENSORS = ("input", "router_probs", "fc1_experts_weights", "fc1_experts_bias", "fc2_experts_weights",
               "fc2_experts_bias", "fc3_experts_weights", "fc3_experts_bias")


def qmoe_moe_attrs_default() -> QmoeMoeAttrs:
    a = QmoeMoeAttrs()
    _lib().qmoe_moe_attrs_default(ctypes.byref(a))
    return a


def make_moe_attrs(attrs: Optional[dict] = None) -> QmoeMoeAttrs:
    """qmoe_moe_attrs from a dict of the README's attribute names."""
    a = qmoe_moe_attrs_default()
    for key, val in (attrs or {}).items():
        if key == "activation_type" and isinstance(val, str):
            val = QMOE_ACT.get(val, 99)
        elif key == "swiglu_limit":
            a.has_swiglu_limit = 0 if val is None else 1
            val = 0.0 if val is None else val
        setattr(a, key, val)
    return a


def _moe_refs(ts, data):
    """Eight tensor arguments in C order from a dict (missing = NULL)."""
    return [_ref(ts.get(n), data) for n in MOE_TENSORS]


def _moe_a(attrs):
    return attrs if isinstance(attrs, QmoeMoeAttrs) else make_moe_attrs(attrs)


def qmoe_moe_validate(tensors: dict, attrs=None, output=None) -> int:
    """Status code of the float MoE contract check.  Arrays may live anywhere."""
    a = _moe_a(attrs)
    return int(_lib().qmoe_moe_validate(*_moe_refs(tensors, False), _ref(output, False), ctypes.byref(a)))


def qmoe_moe_workspace_size(tensors: dict, attrs=None) -> int:
    a = _moe_a(attrs)
    n = ctypes.c_size_t(0)
    st = _lib().qmoe_moe_workspace_size(*_moe_refs(tensors, False), ctypes.byref(a), ctypes.byref(n))
    if st != 0:
        raise QmoeError(st, "qmoe_moe_workspace_size")
    return int(n.value)


def qmoe_moe_forward(tensors: dict, attrs, output, workspace, stream=None, debug: Optional[dict] = None) -> None:
    """Enqueue the float MoE on ``stream``.  ``tensors`` maps the names of
    MOE_TENSORS to contiguous device tensors (optional ones may be absent);
    ``debug`` as for qmoe_forward."""
    a = _moe_a(attrs)
    wptr = workspace.data_ptr() if workspace is not None and workspace.numel() > 0 else None
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = [*_moe_refs(tensors, True), ctypes.byref(a), _ref(output, True), ctypes.c_void_p(wptr),
            ctypes.c_size_t(wbytes), _stream_handle(stream)]
    if debug is None:
        st = _lib().qmoe_moe_forward(*args)
        where = "qmoe_moe_forward"
    else:
        dbg = QmoeDebug()
        for f in ("topk_idx", "topk_w", "counts", "offsets", "perm"):
            t = debug.get(f)
            setattr(dbg, f, t.data_ptr() if t is not None and t.numel() > 0 else None)
        for i, ev in enumerate(debug.get("events") or ()):
            dbg.events[i] = ev
        st = _lib().qmoe_moe_forward_debug(*args, ctypes.byref(dbg))
        where = "qmoe_moe_forward_debug"
    if st != 0:
        raise QmoeError(st, where)


qmoe_moe_forward_debug = qmoe_moe_forward


def moe_forward(tensors: dict, attrs=None, stream=None, workspace=None, output=None, debug=None):
    """Allocate output (and workspace unless given) with torch, then qmoe_moe_forward."""
    import torch
    x = tensors["input"]
    if output is None:
        output = torch.empty_like(x)
    need = qmoe_moe_workspace_size(tensors, attrs)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    qmoe_moe_forward(tensors, attrs, output, workspace, stream, debug)
    return output


# ------------------------------------------------------------------ steps of a routed layer
# These calls are small next to their launches, so their arguments are packed
# at once: every tensor's qmoe_tensor lies in one buffer per thread, which the
# library reads during the call only.
_ONE = struct.Struct("=qiiqqq").pack_into
_CODES = {"float32": QMOE_F32, "uint8": QMOE_U8, "int32": QMOE_I32, "int64": QMOE_I64, "float16": QMOE_F16,
          "bfloat16": QMOE_BF16, "float64": QMOE_F64, "float8_e4m3fn": QMOE_E4M3}
_code_of = {}  # torch dtype -> code, filled as types are met
_tls = threading.local()


def _type_code(dtype):
    return _CODES.get(str(dtype).replace("torch.", ""), 0)


def _pack(ts, first=0):
    """Addresses (None for None) of the tensors' descriptors in this thread's
    buffer from place ``first`` on, valid until its next _pack of that place."""
    buf = getattr(_tls, "buf", None)
    if buf is None:
        buf = _tls.buf = ctypes.create_string_buffer(40 * 16)
        _tls.at = ctypes.addressof(buf)
    at, off, out = _tls.at, 40 * first, []
    for t in ts:
        if t is None:
            out.append(None)
        else:
            dt = t.dtype
            code = _code_of.get(dt)
            if code is not None or hasattr(t, "data_ptr"):
                if code is None:
                    code = _code_of[dt] = _type_code(dt)
                if not t.is_contiguous():
                    raise ValueError("qmoe tensors must be contiguous")
                ptr = t.data_ptr()
            else:  # an array of another kind: extents and type only
                code, ptr = _type_code(dt), 0
            shape = t.shape
            r = len(shape)
            if r == 2:
                d0, d1 = shape
                _ONE(buf, off, ptr, code, 2, d0, d1, 0)
            else:
                d = tuple(shape[:3]) + (0, 0, 0)
                _ONE(buf, off, ptr, code, r, d[0], d[1], d[2])
            out.append(at + off)
        off += 40
    return out


class _Stream:
    """The device of a call's tensors made current, and ``stream`` torch's
    stream, so that what torch allocates belongs to the stream that the work
    runs on."""

    def __init__(self, device, stream):
        import torch
        self.ctx = [torch.cuda.device(device)] + ([] if stream is None else [torch.cuda.stream(stream)])

    def __enter__(self):
        for c in self.ctx:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.ctx):
            c.__exit__(*exc)


_NOTHING = contextlib.nullcontext()


@functools.cache
def _current():
    """(current device's index, handle of a device's current stream): the handle
    straight from torch where it offers that, without the 1 us that building a
    Stream object takes of a 10 us call."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_device, raw or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _on(stream, ts):
    """(context, stream handle) of a call on these tensors, which lie on one
    GPU: its current stream unless ``stream`` is given."""
    dev = None
    for t in ts:
        if t is not None:
            d = t.get_device()
            if dev is None:
                dev = d
            if d != dev or d < 0:
                raise ValueError("qmoe tensors must be on one GPU, got "
                                 f"{sorted({str(u.device) for u in ts if u is not None})}")
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"stream of {stream.device}, tensors on cuda:{dev}")
    device, handle = _current()
    ctx = _NOTHING if stream is None and dev == device() else _Stream(dev, stream)
    return ctx, handle(dev) if stream is None else stream.cuda_stream


def _ok(status, where):
    if status != 0:
        raise QmoeError(status, where)


def _ws(workspace, need, like):
    """(pointer, bytes, tensor to keep until the call is enqueued) of a
    workspace of ``need`` bytes: the one given if it is large enough."""
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        if need == 0:
            return None, 0, None
        workspace = like.new_empty(need, dtype=_uint8())
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _uint8():
    import torch
    return torch.uint8


def _route_args(attrs):
    if isinstance(attrs, dict):
        r = attrs.get("routing", "qmoe")
        return (attrs.get("k", 1), QMOE_ROUTING.get(r, 99) if isinstance(r, str) else r,
                attrs.get("normalize_routing_weights", 0))
    a = make_attrs() if attrs is None else attrs
    return a.k, a.routing, a.normalize_routing_weights


def qmoe_route(router_probs, attrs, indices, weights, stream=None) -> None:
    """Enqueue the routing weights: ``attrs`` holds k, routing and
    normalize_routing_weights (those of ``forward``); indices int32 and
    weights float32, both [T, k]."""
    route(router_probs, attrs, stream, indices, weights)


def route(router_probs, attrs=None, stream=None, indices=None, weights=None):
    """Allocate what is not given, then qmoe_route: (indices, weights)."""
    import torch
    k, routing, norm = _route_args(attrs)
    ctx, st = _on(stream, (router_probs, indices, weights))
    with ctx:
        if indices is None:
            indices = router_probs.new_empty((router_probs.shape[0], max(int(k), 0)), dtype=torch.int32)
        if weights is None:
            weights = router_probs.new_empty(indices.shape, dtype=torch.float32)
        p, i, w = _pack((router_probs, indices, weights))
        _ok(_lib().qmoe_route(p, k, routing, norm, i, w, st), "qmoe_route")
    return indices, weights


def qmoe_route_backward(grad_weights, router_probs, indices, attrs, grad_router_probs, stream=None) -> None:
    """Enqueue the gradient of qmoe_route at the logits (attrs: routing and
    normalize_routing_weights; k is indices' second extent)."""
    route_backward(grad_weights, router_probs, indices, attrs, stream, grad_router_probs)


def route_backward(grad_weights, router_probs, indices, attrs=None, stream=None, grad_router_probs=None):
    """Allocate grad_router_probs [T, E] unless given, then qmoe_route_backward."""
    import torch
    _, routing, norm = _route_args(attrs)
    ctx, st = _on(stream, (grad_weights, router_probs, indices, grad_router_probs))
    with ctx:
        if grad_router_probs is None:
            grad_router_probs = torch.empty_like(router_probs)
        g, p, i, o = _pack((grad_weights, router_probs, indices, grad_router_probs))
        _ok(_lib().qmoe_route_backward(g, p, i, routing, norm, o, st), "qmoe_route_backward")
    return grad_router_probs


def qmoe_dispatch_workspace_size(input, indices, experts) -> int:
    """Workspace bytes of qmoe_dispatch.  Arrays may live anywhere."""
    n = ctypes.c_size_t(0)
    _ok(_lib().qmoe_dispatch_workspace_size(*_refs(input, indices), int(experts), ctypes.byref(n)),
        "qmoe_dispatch_workspace_size")
    return n.value


def qmoe_dispatch(input, indices, experts, rows, offsets, perm, inverse, workspace=None, stream=None) -> None:
    """Enqueue the sort of the slots by expert and the copy of their tokens'
    rows; ``perm`` may be None, ``workspace`` too when its size is 0."""
    ctx, st = _on(stream, (input, indices, rows, offsets, perm, inverse, workspace))
    with ctx:
        w, n, _keep = _ws(workspace, 0, input)
        x, i, r, o, p, v = _pack((input, indices, rows, offsets, perm, inverse))
        _ok(_lib().qmoe_dispatch(x, i, int(experts), r, o, p, v, w, n, st), "qmoe_dispatch")


def dispatch(input, indices, experts, stream=None, workspace=None):
    """Allocate and qmoe_dispatch: (rows [T k, H], offsets [experts + 1], perm [T k], inverse [T, k])."""
    import torch
    ctx, st = _on(stream, (input, indices, workspace))
    with ctx:
        lib = _lib()
        need = ctypes.c_size_t(0)
        x, i = _pack((input, indices))
        _ok(lib.qmoe_dispatch_workspace_size(x, i, int(experts), ctypes.byref(need)), "qmoe_dispatch_workspace_size")
        T, k = indices.shape
        rows = input.new_empty((T * k, input.shape[1]))
        offsets = indices.new_empty(experts + 1, dtype=torch.int32)
        perm = indices.new_empty(T * k, dtype=torch.int32)
        inverse = indices.new_empty((T, k), dtype=torch.int32)
        w, n, _keep = _ws(workspace, need.value, input)
        r, o, p, v = _pack((rows, offsets, perm, inverse), 2)
        _ok(lib.qmoe_dispatch(x, i, int(experts), r, o, p, v, w, n, st), "qmoe_dispatch")
    return rows, offsets, perm, inverse


def qmoe_dispatch_backward(grad_rows, inverse, grad_input, stream=None) -> None:
    """Enqueue the gradient of qmoe_dispatch at its input."""
    dispatch_backward(grad_rows, inverse, stream, grad_input)


def dispatch_backward(grad_rows, inverse, stream=None, grad_input=None):
    """Allocate grad_input [T, H] unless given, then qmoe_dispatch_backward."""
    ctx, st = _on(stream, (grad_rows, inverse, grad_input))
    with ctx:
        if grad_input is None:
            grad_input = grad_rows.new_empty((inverse.shape[0], grad_rows.shape[1]))
        g, v, o = _pack((grad_rows, inverse, grad_input))
        _ok(_lib().qmoe_dispatch_backward(g, v, o, st), "qmoe_dispatch_backward")
    return grad_input


def qmoe_combine(rows, inverse, weights, output, stream=None) -> None:
    """Enqueue the weighted sum of each token's rows (weights None: 1)."""
    combine(rows, inverse, weights, stream, output)


def combine(rows, inverse, weights=None, stream=None, output=None):
    """Allocate output [T, H] unless given, then qmoe_combine."""
    ctx, st = _on(stream, (rows, inverse, weights, output))
    with ctx:
        if output is None:
            output = rows.new_empty((inverse.shape[0], rows.shape[1]))
        r, v, w, o = _pack((rows, inverse, weights, output))
        _ok(_lib().qmoe_combine(r, v, w, o, st), "qmoe_combine")
    return output


def qmoe_combine_backward(grad_output, rows, inverse, weights, grad_rows, grad_weights, stream=None) -> None:
    """Enqueue the gradients of qmoe_combine (either may be None)."""
    ctx, st = _on(stream, (grad_output, rows, inverse, weights, grad_rows, grad_weights))
    with ctx:
        _ok(_lib().qmoe_combine_backward(*_pack((grad_output, rows, inverse, weights, grad_rows, grad_weights)), st),
            "qmoe_combine_backward")


def combine_backward(grad_output, rows, inverse, weights, stream=None):
    """Allocate and qmoe_combine_backward: (grad_rows, grad_weights)."""
    import torch
    ctx, st = _on(stream, (grad_output, rows, inverse, weights))
    with ctx:
        grad_rows, grad_weights = torch.empty_like(rows), torch.empty_like(weights)
        _ok(_lib().qmoe_combine_backward(*_pack((grad_output, rows, inverse, weights, grad_rows, grad_weights)), st),
            "qmoe_combine_backward")
    return grad_rows, grad_weights


# ------------------------------------------------------------------ linear layers
def qmoe_linear_attrs_default() -> QmoeLinearAttrs:
    a = QmoeLinearAttrs()
    _lib().qmoe_linear_attrs_default(ctypes.byref(a))
    return a


def make_linear_attrs(attrs: Optional[dict] = None) -> QmoeLinearAttrs:
    """qmoe_linear_attrs from a dict of the float MoE's attribute names."""
    a = QmoeLinearAttrs(QMOE_ACT["identity"], 0, 1.0, 0.0, 0, 0.0)  # qmoe_linear_attrs_default
    for key, val in (attrs or {}).items():
        if key not in _LINEAR_ATTRS:
            raise ValueError(f"no attribute {key!r} of a linear layer")
        if key == "activation_type" and isinstance(val, str):
            val = QMOE_ACT.get(val, 99)
        elif key == "swiglu_limit":
            a.has_swiglu_limit = 0 if val is None else 1
            val = 0.0 if val is None else val
        setattr(a, key, val)
    return a


_LINEAR_ATTRS = frozenset(f[0] for f in QmoeLinearAttrs._fields_)


def _linear_a(attrs):
    return attrs if isinstance(attrs, QmoeLinearAttrs) else make_linear_attrs(attrs)


def _refs(*ts):
    return [_ref(t, False) for t in ts]


def qmoe_linear_plan_describe(input, weights, offsets=None) -> str:
    """Tiles and ranges of the products of a linear layer and its gradients,
    as one line of text.  Arrays may live anywhere."""
    buf = ctypes.create_string_buffer(128)
    _ok(_lib().qmoe_linear_plan_describe(*_refs(input, weights, offsets), buf, 128), "qmoe_linear_plan_describe")
    return buf.value.decode()


def qmoe_linear_workspace_size(input, weights, bias=None, residual=None, offsets=None, attrs=None, output=None,
                               preact=None) -> int:
    """Workspace bytes of qmoe_linear.  Arrays may live anywhere."""
    a, n = _linear_a(attrs), ctypes.c_size_t(0)
    _ok(_lib().qmoe_linear_workspace_size(*_refs(input, weights, bias, residual, offsets), ctypes.byref(a),
                                          *_refs(output, preact), ctypes.byref(n)), "qmoe_linear_workspace_size")
    return n.value


def qmoe_linear(input, weights, bias, residual, offsets, attrs, output, preact=None, workspace=None,
                stream=None) -> None:
    """Enqueue a linear layer: input [M, K], weights [N, K] or [G, N, K] with
    offsets [G + 1]; bias, residual and preact may be None, workspace too when
    its size is 0."""
    a = _linear_a(attrs)
    ctx, st = _on(stream, (input, weights, bias, residual, offsets, output, preact, workspace))
    with ctx:
        w, n, _keep = _ws(workspace, 0, input)
        t = _pack((input, weights, bias, residual, offsets, output, preact))
        _ok(_lib().qmoe_linear(*t[:5], ctypes.byref(a), t[5], t[6], w, n, st), "qmoe_linear")


def linear(input, weights, bias=None, residual=None, offsets=None, attrs=None, keep_preact=False, stream=None,
           workspace=None, output=None):
    """Allocate output (and preact with ``keep_preact``), then qmoe_linear:
    output, or (output, preact)."""
    a = _linear_a(attrs)
    ctx, st = _on(stream, (input, weights, bias, residual, offsets, workspace, output))
    with ctx:
        M, N = input.shape[0], weights.shape[-2]
        if output is None:
            output = input.new_empty((M, N // 2 if a.activation_type == QMOE_ACT["swiglu"] else N))
        preact = input.new_empty((M, N)) if keep_preact else None
        lib, need, attr = _lib(), ctypes.c_size_t(0), ctypes.byref(a)
        t = _pack((input, weights, bias, residual, offsets, output, preact))
        _ok(lib.qmoe_linear_workspace_size(*t[:5], attr, t[5], t[6], ctypes.byref(need)), "qmoe_linear_workspace_size")
        w, n, _keep = _ws(workspace, need.value, input)
        _ok(lib.qmoe_linear(*t[:5], attr, t[5], t[6], w, n, st), "qmoe_linear")
    return (output, preact) if keep_preact else output


def qmoe_linear_backward_workspace_size(grad_output, input, weights, preact=None, offsets=None, attrs=None,
                                        grad_input=None, grad_weights=None, grad_bias=None) -> int:
    """Workspace bytes of qmoe_linear_backward for the gradients given.  Arrays may live anywhere."""
    a, n = _linear_a(attrs), ctypes.c_size_t(0)
    _ok(_lib().qmoe_linear_backward_workspace_size(
        *_refs(grad_output, input, weights, preact, offsets), ctypes.byref(a),
        *_refs(grad_input, grad_weights, grad_bias), ctypes.byref(n)), "qmoe_linear_backward_workspace_size")
    return n.value


def qmoe_linear_backward(grad_output, input, weights, preact, offsets, attrs, grad_input, grad_weights, grad_bias,
                         workspace=None, stream=None) -> None:
    """Enqueue the gradients of qmoe_linear (any may be None); preact None for
    the identity, offsets None for a dense layer."""
    a = _linear_a(attrs)
    ctx, st = _on(stream, (grad_output, input, weights, preact, offsets, grad_input, grad_weights, grad_bias,
                           workspace))
    with ctx:
        w, n, _keep = _ws(workspace, 0, input)
        t = _pack((grad_output, input, weights, preact, offsets, grad_input, grad_weights, grad_bias))
        _ok(_lib().qmoe_linear_backward(*t[:5], ctypes.byref(a), *t[5:], w, n, st), "qmoe_linear_backward")


def linear_backward(grad_output, input, weights, preact=None, offsets=None, attrs=None, bias=False, stream=None,
                    workspace=None):
    """Allocate and qmoe_linear_backward: (grad_input, grad_weights, grad_bias),
    grad_bias None unless ``bias``."""
    import torch
    a = _linear_a(attrs)
    ctx, st = _on(stream, (grad_output, input, weights, preact, offsets, workspace))
    with ctx:
        gi, gw = torch.empty_like(input), torch.empty_like(weights)
        gb = weights.new_empty(weights.shape[:-1]) if bias else None
        lib, need, attr = _lib(), ctypes.c_size_t(0), ctypes.byref(a)
        t = _pack((grad_output, input, weights, preact, offsets, gi, gw, gb))
        _ok(lib.qmoe_linear_backward_workspace_size(*t[:5], attr, *t[5:], ctypes.byref(need)),
            "qmoe_linear_backward_workspace_size")
        w, n, _keep = _ws(workspace, need.value, input)
        _ok(lib.qmoe_linear_backward(*t[:5], attr, *t[5:], w, n, st), "qmoe_linear_backward")
    return gi, gw, gb


# ------------------------------------------------------------------ rows in 8 bits
def _code_type(format):
    """torch type of the codes of "int8" (uint8, 128 for 0) or "e4m3"."""
    import torch
    if format == "int8":
        return torch.uint8
    if format == "e4m3":
        return torch.float8_e4m3fn
    raise ValueError(f"no 8-bit format {format!r} (int8 or e4m3)")


def _eight(like, format, rows, cols, block_size):
    """Empty codes and scales of rows x cols values."""
    import torch
    blocks = -(-cols // block_size) if block_size > 0 else 0  # (the library refuses other sizes)
    return like.new_empty((rows, cols), dtype=_code_type(format)), like.new_empty((rows, blocks), dtype=torch.float32)


def qmoe_quantize_rows(input, block_size, codes, scales, stream=None) -> None:
    """Enqueue rows to 8 bits: codes [M, N] uint8 or float8_e4m3fn, scales
    [M, ceil(N / block_size)] float32."""
    ctx, st = _on(stream, (input, codes, scales))
    with ctx:
        x, c, s = _pack((input, codes, scales))
        _ok(_lib().qmoe_quantize_rows(x, block_size, c, s, st), "qmoe_quantize_rows")


def quantize_rows(input, format="int8", block_size=128, stream=None):
    """Allocate and qmoe_quantize_rows: (codes, scales); format "int8" or "e4m3"."""
    ctx, st = _on(stream, (input,))
    with ctx:
        codes, scales = _eight(input, format, input.shape[0], input.shape[-1], block_size)
        x, c, s = _pack((input, codes, scales))
        _ok(_lib().qmoe_quantize_rows(x, block_size, c, s, st), "qmoe_quantize_rows")
    return codes, scales


def qmoe_dequantize_rows(codes, scales, block_size, perm, output, stream=None) -> None:
    """Enqueue the values of rows in 8 bits; perm None: row for row."""
    ctx, st = _on(stream, (codes, scales, perm, output))
    with ctx:
        c, s, p, o = _pack((codes, scales, perm, output))
        _ok(_lib().qmoe_dequantize_rows(c, s, block_size, p, o, st), "qmoe_dequantize_rows")


def dequantize_rows(codes, scales, dtype, block_size=128, perm=None, stream=None, output=None):
    """Allocate output of ``dtype`` unless given, then qmoe_dequantize_rows:
    the rows of codes, or with ``perm`` (of qmoe_dispatch) the slots' rows."""
    ctx, st = _on(stream, (codes, scales, perm, output))
    with ctx:
        if output is None:
            rows = codes.shape[0] if perm is None else perm.shape[0]
            output = codes.new_empty((rows, codes.shape[1]), dtype=dtype)
        c, s, p, o = _pack((codes, scales, perm, output))
        _ok(_lib().qmoe_dequantize_rows(c, s, block_size, p, o, st), "qmoe_dequantize_rows")
    return output


# ------------------------------------------------------------------ norm
def qmoe_rms_norm(input, residual, weight, epsilon, sum, output, codes=None, scales=None, block_size=128,
                  stream=None) -> None:
    """Enqueue the root-mean-square norm; residual, weight, sum, output, or
    codes and scales may be None (not output and codes both)."""
    ctx, st = _on(stream, (input, residual, weight, sum, output, codes, scales))
    with ctx:
        x, r, w, h, y, c, s = _pack((input, residual, weight, sum, output, codes, scales))
        _ok(_lib().qmoe_rms_norm(x, r, w, epsilon, h, y, c, s, block_size, st), "qmoe_rms_norm")


def rms_norm(input, weight=None, residual=None, epsilon=1e-6, format=None, block_size=128, keep_output=True,
             stream=None):
    """Allocate and qmoe_rms_norm: (output, sum, codes, scales), sum None
    without residual, codes and scales None without ``format`` ("int8" or
    "e4m3"), output None unless ``keep_output``."""
    import torch
    ctx, st = _on(stream, (input, weight, residual))
    with ctx:
        output = torch.empty_like(input) if keep_output else None
        sum = torch.empty_like(input) if residual is not None else None
        codes = scales = None
        if format is not None:
            codes, scales = _eight(input, format, input.shape[0], input.shape[-1], block_size)
        x, r, w, h, y, c, s = _pack((input, residual, weight, sum, output, codes, scales))
        _ok(_lib().qmoe_rms_norm(x, r, w, epsilon, h, y, c, s, block_size, st), "qmoe_rms_norm")
    return output, sum, codes, scales


def qmoe_rms_norm_backward_workspace_size(grad_output, grad_sum, input, weight, epsilon=1e-6, grad_input=None,
                                          grad_weight=None) -> int:
    """Workspace bytes of qmoe_rms_norm_backward for the gradients given.  Arrays may live anywhere."""
    n = ctypes.c_size_t(0)
    _ok(_lib().qmoe_rms_norm_backward_workspace_size(*_refs(grad_output, grad_sum, input, weight), epsilon,
                                                     *_refs(grad_input, grad_weight), ctypes.byref(n)),
        "qmoe_rms_norm_backward_workspace_size")
    return n.value


def qmoe_rms_norm_backward(grad_output, grad_sum, input, weight, epsilon, grad_input, grad_weight, workspace=None,
                           stream=None) -> None:
    """Enqueue the gradients of qmoe_rms_norm (either may be None); input is the
    forward's sum, or its input where it had no residual."""
    ctx, st = _on(stream, (grad_output, grad_sum, input, weight, grad_input, grad_weight, workspace))
    with ctx:
        w, n, _keep = _ws(workspace, 0, input)
        t = _pack((grad_output, grad_sum, input, weight, grad_input, grad_weight))
        _ok(_lib().qmoe_rms_norm_backward(*t[:4], epsilon, *t[4:], w, n, st), "qmoe_rms_norm_backward")


def rms_norm_backward(grad_output, input, weight=None, grad_sum=None, epsilon=1e-6, stream=None, workspace=None):
    """Allocate and qmoe_rms_norm_backward: (grad_input, grad_weight),
    grad_weight None without weight."""
    import torch
    ctx, st = _on(stream, (grad_output, input, weight, grad_sum, workspace))
    with ctx:
        gi = torch.empty_like(input)
        gw = torch.empty_like(weight) if weight is not None else None
        lib, need = _lib(), ctypes.c_size_t(0)
        t = _pack((grad_output, grad_sum, input, weight, gi, gw))
        _ok(lib.qmoe_rms_norm_backward_workspace_size(*t[:4], epsilon, *t[4:], ctypes.byref(need)),
            "qmoe_rms_norm_backward_workspace_size")
        w, n, _keep = _ws(workspace, need.value, input)
        _ok(lib.qmoe_rms_norm_backward(*t[:4], epsilon, *t[4:], w, n, st), "qmoe_rms_norm_backward")
    return gi, gw


# ------------------------------------------------------------------ routing from scores
_ROUTE_ATTRS = frozenset(f[0] for f in QmoeRouteAttrs._fields_)


def qmoe_route_attrs_default() -> QmoeRouteAttrs:
    a = QmoeRouteAttrs()
    _lib().qmoe_route_attrs_default(ctypes.byref(a))
    return a


def make_route_attrs(attrs: Optional[dict] = None) -> QmoeRouteAttrs:
    """qmoe_route_attrs from a dict of its fields ("scores" also by name)."""
    a = QmoeRouteAttrs(1, QMOE_SCORES["softmax"], 1, 1, 2, 0, 1.0)  # qmoe_route_attrs_default
    for key, val in (attrs or {}).items():
        if key not in _ROUTE_ATTRS:
            raise ValueError(f"no attribute {key!r} of routing from scores")
        if key == "scores" and isinstance(val, str):
            val = QMOE_SCORES.get(val, 99)
        setattr(a, key, val)
    return a


def _scored_a(attrs):
    return attrs if isinstance(attrs, QmoeRouteAttrs) else make_route_attrs(attrs)


def qmoe_route_scored(router_probs, bias, attrs, indices, weights, stream=None) -> None:
    """Enqueue routing from scores; bias may be None, indices int32 and weights
    float32 are [T, k]."""
    route_scored(router_probs, bias, attrs, stream, indices, weights)


def route_scored(router_probs, bias=None, attrs=None, stream=None, indices=None, weights=None):
    """Allocate what is not given, then qmoe_route_scored: (indices, weights)."""
    import torch
    a = _scored_a(attrs)
    ctx, st = _on(stream, (router_probs, bias, indices, weights))
    with ctx:
        if indices is None:
            indices = router_probs.new_empty((router_probs.shape[0], max(a.k, 0)), dtype=torch.int32)
        if weights is None:
            weights = router_probs.new_empty(indices.shape, dtype=torch.float32)
        p, b, i, w = _pack((router_probs, bias, indices, weights))
        _ok(_lib().qmoe_route_scored(p, b, ctypes.byref(a), i, w, st), "qmoe_route_scored")
    return indices, weights


def qmoe_route_scored_backward(grad_weights, router_probs, indices, attrs, grad_router_probs, stream=None) -> None:
    """Enqueue the gradient of qmoe_route_scored at the logits (k is indices'
    second extent)."""
    route_scored_backward(grad_weights, router_probs, indices, attrs, stream, grad_router_probs)


def route_scored_backward(grad_weights, router_probs, indices, attrs=None, stream=None, grad_router_probs=None):
    """Allocate grad_router_probs [T, E] unless given, then qmoe_route_scored_backward."""
    import torch
    a = _scored_a(attrs)
    ctx, st = _on(stream, (grad_weights, router_probs, indices, grad_router_probs))
    with ctx:
        if grad_router_probs is None:
            grad_router_probs = torch.empty_like(router_probs)
        g, p, i, o = _pack((grad_weights, router_probs, indices, grad_router_probs))
        _ok(_lib().qmoe_route_scored_backward(g, p, i, ctypes.byref(a), o, st), "qmoe_route_scored_backward")
    return grad_router_probs


# ------------------------------------------------------------------ linear layers and their checkpoints
def _pair(t):
    """(tensor, None), or (codes, scales) of what is held in 8 bits."""
    return t if isinstance(t, (tuple, list)) else (t, None)


def qmoe_linear_q8_workspace_size(input, weights, bias=None, residual=None, offsets=None, attrs=None, output=None,
                                  codes=None, scales=None, block_size=128) -> int:
    """Workspace bytes of qmoe_linear_q8.  Arrays may live anywhere."""
    a, n = _linear_a(attrs), ctypes.c_size_t(0)
    _ok(_lib().qmoe_linear_q8_workspace_size(*_refs(input, weights, bias, residual, offsets), ctypes.byref(a),
                                             *_refs(output, codes, scales), block_size, ctypes.byref(n)),
        "qmoe_linear_q8_workspace_size")
    return n.value


def qmoe_linear_q8(input, weights, bias, residual, offsets, attrs, output, codes, scales, block_size=128,
                   workspace=None, stream=None) -> None:
    """Enqueue a linear layer whose pre-activations [M, N] leave in 8 bits; the
    rest as qmoe_linear."""
    a = _linear_a(attrs)
    ctx, st = _on(stream, (input, weights, bias, residual, offsets, output, codes, scales, workspace))
    with ctx:
        w, n, _keep = _ws(workspace, 0, input)
        t = _pack((input, weights, bias, residual, offsets, output, codes, scales))
        _ok(_lib().qmoe_linear_q8(*t[:5], ctypes.byref(a), *t[5:], block_size, w, n, st), "qmoe_linear_q8")


def linear_q8(input, weights, bias=None, residual=None, offsets=None, attrs=None, format="int8", block_size=128,
              stream=None, workspace=None, output=None):
    """Allocate and qmoe_linear_q8: (output, codes, scales)."""
    a = _linear_a(attrs)
    ctx, st = _on(stream, (input, weights, bias, residual, offsets, workspace, output))
    with ctx:
        M, N = input.shape[0], weights.shape[-2]
        if output is None:
            output = input.new_empty((M, N // 2 if a.activation_type == QMOE_ACT["swiglu"] else N))
        codes, scales = _eight(input, format, M, N, block_size)
        lib, need, attr = _lib(), ctypes.c_size_t(0), ctypes.byref(a)
        t = _pack((input, weights, bias, residual, offsets, output, codes, scales))
        _ok(lib.qmoe_linear_q8_workspace_size(*t[:5], attr, *t[5:], block_size, ctypes.byref(need)),
            "qmoe_linear_q8_workspace_size")
        w, n, _keep = _ws(workspace, need.value, input)
        _ok(lib.qmoe_linear_q8(*t[:5], attr, *t[5:], block_size, w, n, st), "qmoe_linear_q8")
    return output, codes, scales


def qmoe_linear_backward_q8_workspace_size(grad_output, input, weights, preact=None, offsets=None, attrs=None,
                                           grad_input=None, grad_weights=None, grad_bias=None, block_size=128,
                                           perm=None) -> int:
    """Workspace bytes of qmoe_linear_backward_q8 for the gradients given; input
    and preact tensors or (codes, scales).  Arrays may live anywhere."""
    a, n = _linear_a(attrs), ctypes.c_size_t(0)
    (x, xs), (z, zs) = _pair(input), _pair(preact)
    _ok(_lib().qmoe_linear_backward_q8_workspace_size(
        *_refs(grad_output, x, xs, perm, weights, z, zs), block_size, *_refs(offsets), ctypes.byref(a),
        *_refs(grad_input, grad_weights, grad_bias), ctypes.byref(n)), "qmoe_linear_backward_q8_workspace_size")
    return n.value


def qmoe_linear_backward_q8(grad_output, input, weights, preact, offsets, attrs, grad_input, grad_weights, grad_bias,
                            block_size=128, perm=None, workspace=None, stream=None) -> None:
    """Enqueue the gradients of qmoe_linear from an input and pre-activations
    that are each a tensor or (codes, scales); with ``perm`` the input's codes
    are held once a token.  The rest as qmoe_linear_backward."""
    a = _linear_a(attrs)
    (x, xs), (z, zs) = _pair(input), _pair(preact)
    ctx, st = _on(stream, (grad_output, x, xs, perm, weights, z, zs, offsets, grad_input, grad_weights, grad_bias,
                           workspace))
    with ctx:
        w, n, _keep = _ws(workspace, 0, weights)
        t = _pack((grad_output, x, xs, perm, weights, z, zs, offsets, grad_input, grad_weights, grad_bias))
        _ok(_lib().qmoe_linear_backward_q8(*t[:7], block_size, t[7], ctypes.byref(a), *t[8:], w, n, st),
            "qmoe_linear_backward_q8")


def linear_backward_q8(grad_output, input, weights, preact=None, offsets=None, attrs=None, bias=False, block_size=128,
                       perm=None, stream=None, workspace=None):
    """Allocate and qmoe_linear_backward_q8: (grad_input, grad_weights,
    grad_bias), grad_bias None unless ``bias``."""
    import torch
    a = _linear_a(attrs)
    (x, xs), (z, zs) = _pair(input), _pair(preact)
    ctx, st = _on(stream, (grad_output, x, xs, perm, weights, z, zs, offsets, workspace))
    with ctx:
        gi = weights.new_empty((grad_output.shape[0], weights.shape[-1]))
        gw = torch.empty_like(weights)
        gb = weights.new_empty(weights.shape[:-1]) if bias else None
        lib, need, attr = _lib(), ctypes.c_size_t(0), ctypes.byref(a)
        t = _pack((grad_output, x, xs, perm, weights, z, zs, offsets, gi, gw, gb))
        _ok(lib.qmoe_linear_backward_q8_workspace_size(*t[:7], block_size, t[7], attr, *t[8:], ctypes.byref(need)),
            "qmoe_linear_backward_q8_workspace_size")
        w, n, _keep = _ws(workspace, need.value, weights)
        _ok(lib.qmoe_linear_backward_q8(*t[:7], block_size, t[7], attr, *t[8:], w, n, st), "qmoe_linear_backward_q8")
    return gi, gw, gb
