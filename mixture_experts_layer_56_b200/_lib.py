"""ctypes binding of libmoe.so (include/moe.h): argument marshalling only.

Every function below has the name of the C entry point it calls; tensors are
passed as device (or host) pointers, ``None`` as NULL, and the stream defaults
to torch's current CUDA stream.  A non-zero status raises ``MoeError``.
Loading fails loudly when the library has not been built: there is no other
implementation behind these names.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_char_p, c_int, c_int32, c_int64, c_size_t, c_uint64, c_void_p

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_DTYPE_F32 = 0
MOE_DTYPE_BF16 = 1
MOE_FLAG_BIAS_SELECT_ONLY = 1
MOE_FLAG_GEMM_SINGLE_CTA = 2
MOE_FLAG_GEMM_CTA_PAIR = 4
MOE_FLAG_ROUTER_SIMT = 8
MOE_FLAG_INJECT_WAIT_TIMEOUT = 16
MOE_FLAG_GEMM_NARROW = 32

MOE_OK = 0
MOE_ERR_NULLPTR = -1
MOE_ERR_SHAPE = -2
MOE_ERR_ALIGN = -3
MOE_ERR_WORKSPACE = -4
MOE_ERR_DTYPE = -5
MOE_ERR_CUDA = -6
MOE_ERR_DEVICE_CHECK = -7
MOE_ERR_UNSUPPORTED = -8
MOE_ERR_SCRATCH_LIMIT = -9

# stage kinds of the tracer (include/moe.h MOE_KERNEL_*)
MOE_KERNEL_ROUTER = 1
MOE_KERNEL_DISPATCH = 2
MOE_KERNEL_GATHER = 3
MOE_KERNEL_GEMM_GATE_UP = 4
MOE_KERNEL_GEMM_DOWN = 5
MOE_KERNEL_COMBINE = 6
MOE_KERNEL_FFN_F32 = 7
MOE_KERNEL_MEMSET = 8
MOE_KERNEL_PACK = 9
MOE_KERNEL_BALANCE = 10
MOE_KERNEL_DECODE_LAYER = 11
MOE_KERNEL_GROUPED_FWD = 12
MOE_KERNEL_GROUPED_DX = 13
MOE_KERNEL_GROUPED_DW = 14
MOE_KERNEL_SWIGLU = 15
MOE_KERNEL_SWIGLU_BACKWARD = 16
MOE_KERNEL_LAYER_NORM = 17
MOE_KERNEL_LAYER_NORM_BACKWARD = 18
MOE_KERNEL_ORTHOGONALIZE = 19
MOE_GROUPED_DW_F32 = 1
MOE_GROUPED_DW_ACCUMULATE = 2
MOE_PATH_STAGES = 0
MOE_PATH_DECODE_LAYER = 1
MOE_PATH_SMALL_BATCH = 2
MOE_DISPATCH_STATIC_SCRATCH_BYTES = 512 * 1024


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {code} ({strerror(code)})")


class MoeShape(ctypes.Structure):
    _fields_ = [("T", c_int64), ("d", c_int32), ("n_routed", c_int32), ("n_shared", c_int32),
                ("inter", c_int32), ("top_k", c_int32), ("dtype", c_int32), ("flags", c_int32)]

    def __repr__(self):
        return (f"MoeShape(T={self.T}, d={self.d}, n_routed={self.n_routed}, "
                f"n_shared={self.n_shared}, inter={self.inter}, top_k={self.top_k}, "
                f"dtype={self.dtype}, flags={self.flags})")


class MoeGroupedShape(ctypes.Structure):
    _fields_ = [("rows", c_int64), ("n_groups", c_int32), ("n", c_int32), ("k", c_int32),
                ("dtype", c_int32), ("flags", c_int32)]


class MoeSwigluShape(ctypes.Structure):
    _fields_ = [("rows", c_int64), ("inter", c_int32), ("dtype", c_int32)]


class MoeNormShape(ctypes.Structure):
    _fields_ = [("T", c_int64), ("d", c_int32), ("dtype", c_int32), ("eps", ctypes.c_float)]


class MoeOrthoShape(ctypes.Structure):
    _fields_ = [("n_mats", c_int32), ("rows", c_int32), ("cols", c_int32), ("steps", c_int32),
                ("dtype", c_int32)]


_SHAPE = POINTER(MoeShape)
_GROUPED = POINTER(MoeGroupedShape)
_SWIGLU = POINTER(MoeSwigluShape)
_NORM = POINTER(MoeNormShape)
_ORTHO = POINTER(MoeOrthoShape)
_V = c_void_p

# name -> (restype, argtypes)
SIGNATURES = {
    "moe_strerror": (c_char_p, [c_int]),
    "moe_version": (c_char_p, []),
    "moe_launch_count": (c_uint64, []),
    "moe_workspace_size": (c_int, [_SHAPE, POINTER(c_size_t)]),
    "moe_workspace_size_host": (c_int, [_SHAPE, POINTER(c_size_t)]),
    "moe_forward_path": (c_int, [_SHAPE, POINTER(c_int32)]),
    "moe_pack_w13": (c_int, [_SHAPE, c_int32, _V, _V, _V, _V]),
    "moe_route": (c_int, [_SHAPE, _V, _V, _V, _V, _V, _V]),
    "moe_dispatch": (c_int, [_SHAPE, _V, _V, _V, _V, _V, _V, c_size_t, _V]),
    "moe_dispatch_static_scratch": (c_int, [_SHAPE, _V, _V, _V, _V, _V, _V]),
    "moe_expert_ffn": (c_int, [_SHAPE, _V, _V, _V, _V, _V, _V, _V, _V, _V, _V, c_size_t, _V]),
    "moe_combine": (c_int, [_SHAPE, _V, _V, _V, _V, _V, _V, _V]),
    "moe_layer_forward": (c_int, [_SHAPE, _V, _V, _V, _V, _V, _V, _V, _V, _V, c_size_t, _V]),
    "moe_layer_forward_host": (c_int, [_SHAPE, _V, _V, _V, _V, _V, _V, _V, _V, _V, c_size_t, _V]),
    "moe_expert_balance": (c_int, [_SHAPE, _V, _V, _V, _V, _V, _V, _V, c_size_t, _V]),
    "moe_grouped_workspace_size": (c_int, [_GROUPED, POINTER(c_size_t)]),
    "moe_grouped_matmul": (c_int, [_GROUPED, _V, _V, _V, _V, _V, c_size_t, _V]),
    "moe_grouped_matmul_dx": (c_int, [_GROUPED, _V, _V, _V, _V, _V, c_size_t, _V]),
    "moe_grouped_matmul_dw": (c_int, [_GROUPED, _V, _V, _V, _V, _V, c_size_t, _V]),
    "moe_swiglu": (c_int, [_SWIGLU, _V, _V, _V]),
    "moe_swiglu_backward": (c_int, [_SWIGLU, _V, _V, _V, _V]),
    "moe_layer_norm": (c_int, [_NORM, _V, _V, _V, _V, _V, _V, _V]),
    "moe_layer_norm_workspace_size": (c_int, [_NORM, POINTER(c_size_t)]),
    "moe_layer_norm_backward": (c_int, [_NORM, _V, _V, _V, _V, _V, _V, _V, _V, _V, c_size_t, _V]),
    "moe_orthogonalize_workspace_size": (c_int, [_ORTHO, POINTER(c_size_t)]),
    "moe_orthogonalize": (c_int, [_ORTHO, POINTER(ctypes.c_float), _V, _V, _V, c_size_t, _V]),
    "moe_read_status": (c_int, [_V, POINTER(c_int32), _V]),
    "moe_profile_enable": (c_int, [c_int]),
    "moe_profile_read": (c_int, [POINTER(c_int32), POINTER(ctypes.c_float), c_int32,
                                 POINTER(c_int32)]),
    "moe_kernel_name": (c_char_p, [c_int32]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if libmoe.so is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m mixture_experts_layer_56_b200.build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(h, name)
            f.restype = res
            f.argtypes = args
        _lib = h
    return _lib


def strerror(code: int) -> str:
    return lib().moe_strerror(code).decode()


def _ptr(x):
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


_current_raw_stream = None


def _stream(stream):
    if stream is None:
        global _current_raw_stream
        if _current_raw_stream is None:
            import torch
            raw, device = (getattr(torch._C, n, None)
                           for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
            if raw is not None and device is not None:
                # current_stream() without its Stream object, which costs more
                # than a small kernel takes to launch
                torch.cuda.init()
                _current_raw_stream = lambda: raw(device())  # noqa: E731
            else:
                _current_raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        return _current_raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, rc):
    if rc != MOE_OK:
        raise MoeError(fn, rc)
    return rc


def make_shape(T, d, n_routed, n_shared, inter, top_k, dtype=MOE_DTYPE_BF16, flags=0) -> MoeShape:
    return MoeShape(T, d, n_routed, n_shared, inter, top_k, dtype, flags)


# ------------------------------------------------------------- entry points
def moe_version() -> str:
    return lib().moe_version().decode()


def moe_launch_count() -> int:
    return int(lib().moe_launch_count())


def moe_workspace_size(shape: MoeShape) -> int:
    n = c_size_t(0)
    _check("moe_workspace_size", lib().moe_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def moe_workspace_size_host(shape: MoeShape) -> int:
    n = c_size_t(0)
    _check("moe_workspace_size_host",
           lib().moe_workspace_size_host(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def moe_forward_path(shape: MoeShape) -> int:
    p = c_int32(0)
    _check("moe_forward_path", lib().moe_forward_path(ctypes.byref(shape), ctypes.byref(p)))
    return p.value


def moe_pack_w13(shape, n_experts, W1, W3, W13, stream=None):
    return _check("moe_pack_w13", lib().moe_pack_w13(
        ctypes.byref(shape), n_experts, _ptr(W1), _ptr(W3), _ptr(W13), _stream(stream)))


def moe_route(shape, u, E, bias, idx, w, stream=None):
    return _check("moe_route", lib().moe_route(
        ctypes.byref(shape), _ptr(u), _ptr(E), _ptr(bias), _ptr(idx), _ptr(w), _stream(stream)))


def moe_dispatch(shape, idx, counts, offsets, perm, inv, ws, ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    return _check("moe_dispatch", lib().moe_dispatch(
        ctypes.byref(shape), _ptr(idx), _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv),
        _ptr(ws), nb, _stream(stream)))


def moe_dispatch_static_scratch(shape, idx, counts, offsets, perm, inv, stream=None):
    return _check("moe_dispatch_static_scratch", lib().moe_dispatch_static_scratch(
        ctypes.byref(shape), _ptr(idx), _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv),
        _stream(stream)))


def moe_expert_ffn(shape, u, perm, offsets, W13, W2, W13_s, W2_s, y, ysh, ws, ws_bytes=None,
                   stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    return _check("moe_expert_ffn", lib().moe_expert_ffn(
        ctypes.byref(shape), _ptr(u), _ptr(perm), _ptr(offsets), _ptr(W13), _ptr(W2),
        _ptr(W13_s), _ptr(W2_s), _ptr(y), _ptr(ysh), _ptr(ws), nb, _stream(stream)))


def moe_combine(shape, u, ysh, y, w, inv, h, stream=None):
    return _check("moe_combine", lib().moe_combine(
        ctypes.byref(shape), _ptr(u), _ptr(ysh), _ptr(y), _ptr(w), _ptr(inv), _ptr(h),
        _stream(stream)))


def moe_layer_forward(shape, u, E, bias, W13, W2, W13_s, W2_s, h, ws, ws_bytes=None,
                      stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    return _check("moe_layer_forward", lib().moe_layer_forward(
        ctypes.byref(shape), _ptr(u), _ptr(E), _ptr(bias), _ptr(W13), _ptr(W2), _ptr(W13_s),
        _ptr(W2_s), _ptr(h), _ptr(ws), nb, _stream(stream)))


def moe_layer_forward_host(shape, u_host, E, bias, W13, W2, W13_s, W2_s, h_host, ws,
                           ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    return _check("moe_layer_forward_host", lib().moe_layer_forward_host(
        ctypes.byref(shape), _ptr(u_host), _ptr(E), _ptr(bias), _ptr(W13), _ptr(W2),
        _ptr(W13_s), _ptr(W2_s), _ptr(h_host), _ptr(ws), nb, _stream(stream)))


def moe_expert_balance(shape, u, E, bias, counts, f, P, ws, ws_bytes=None, stream=None):
    nb = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    return _check("moe_expert_balance", lib().moe_expert_balance(
        ctypes.byref(shape), _ptr(u), _ptr(E), _ptr(bias), _ptr(counts), _ptr(f), _ptr(P),
        _ptr(ws), nb, _stream(stream)))


# ------------------------------------------------------- training operators
def make_grouped_shape(rows, n_groups, n, k, dtype=MOE_DTYPE_BF16, flags=0) -> MoeGroupedShape:
    return MoeGroupedShape(rows, n_groups, n, k, dtype, flags)


def make_swiglu_shape(rows, inter, dtype=MOE_DTYPE_BF16) -> MoeSwigluShape:
    return MoeSwigluShape(rows, inter, dtype)


def make_norm_shape(T, d, dtype=MOE_DTYPE_BF16, eps=1e-5) -> MoeNormShape:
    return MoeNormShape(T, d, dtype, eps)


def make_ortho_shape(n_mats, rows, cols, steps=5, dtype=MOE_DTYPE_BF16) -> MoeOrthoShape:
    return MoeOrthoShape(n_mats, rows, cols, steps, dtype)


def _size(fn, shape) -> int:
    n = c_size_t(0)
    _check(fn, getattr(lib(), fn)(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def moe_grouped_workspace_size(shape: MoeGroupedShape) -> int:
    return _size("moe_grouped_workspace_size", shape)


def moe_layer_norm_workspace_size(shape: MoeNormShape) -> int:
    return _size("moe_layer_norm_workspace_size", shape)


def moe_orthogonalize_workspace_size(shape: MoeOrthoShape) -> int:
    return _size("moe_orthogonalize_workspace_size", shape)


def _ws_bytes(ws, ws_bytes):
    return ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes


def moe_grouped_matmul(shape, X, offsets, W, Y, ws, ws_bytes=None, stream=None):
    return _check("moe_grouped_matmul", lib().moe_grouped_matmul(
        ctypes.byref(shape), _ptr(X), _ptr(offsets), _ptr(W), _ptr(Y), _ptr(ws),
        _ws_bytes(ws, ws_bytes), _stream(stream)))


def moe_grouped_matmul_dx(shape, dY, offsets, W, dX, ws, ws_bytes=None, stream=None):
    return _check("moe_grouped_matmul_dx", lib().moe_grouped_matmul_dx(
        ctypes.byref(shape), _ptr(dY), _ptr(offsets), _ptr(W), _ptr(dX), _ptr(ws),
        _ws_bytes(ws, ws_bytes), _stream(stream)))


def moe_grouped_matmul_dw(shape, dY, X, offsets, dW, ws, ws_bytes=None, stream=None):
    return _check("moe_grouped_matmul_dw", lib().moe_grouped_matmul_dw(
        ctypes.byref(shape), _ptr(dY), _ptr(X), _ptr(offsets), _ptr(dW), _ptr(ws),
        _ws_bytes(ws, ws_bytes), _stream(stream)))


def moe_swiglu(shape, gu, a, stream=None):
    return _check("moe_swiglu", lib().moe_swiglu(ctypes.byref(shape), _ptr(gu), _ptr(a),
                                                 _stream(stream)))


def moe_swiglu_backward(shape, gu, da, dgu, stream=None):
    return _check("moe_swiglu_backward", lib().moe_swiglu_backward(
        ctypes.byref(shape), _ptr(gu), _ptr(da), _ptr(dgu), _stream(stream)))


def moe_layer_norm(shape, x, gamma, beta, y, mean, rstd, stream=None):
    return _check("moe_layer_norm", lib().moe_layer_norm(
        ctypes.byref(shape), _ptr(x), _ptr(gamma), _ptr(beta), _ptr(y), _ptr(mean), _ptr(rstd),
        _stream(stream)))


def moe_layer_norm_backward(shape, dy, x, gamma, mean, rstd, dx, dgamma, dbeta, ws, ws_bytes=None,
                            stream=None):
    return _check("moe_layer_norm_backward", lib().moe_layer_norm_backward(
        ctypes.byref(shape), _ptr(dy), _ptr(x), _ptr(gamma), _ptr(mean), _ptr(rstd), _ptr(dx),
        _ptr(dgamma), _ptr(dbeta), _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream)))


def moe_orthogonalize(shape, M, O, ws, ws_bytes=None, coef=None, stream=None):
    """`coef`: 3 * shape.steps host floats (a, b, c per step), or None for
    the library's own."""
    if coef is not None:
        coef = [float(c) for c in coef]
        if len(coef) != 3 * shape.steps:
            raise ValueError(f"coef holds {len(coef)} numbers, not 3 * {shape.steps}")
        coef = (ctypes.c_float * len(coef))(*coef)
    return _check("moe_orthogonalize", lib().moe_orthogonalize(
        ctypes.byref(shape), coef, _ptr(M), _ptr(O), _ptr(ws), _ws_bytes(ws, ws_bytes),
        _stream(stream)))


def moe_read_status(ws, stream=None) -> int:
    st = c_int32(0)
    _check("moe_read_status", lib().moe_read_status(_ptr(ws), ctypes.byref(st), _stream(stream)))
    return st.value


def moe_profile_enable(on=True, kinds=None):
    """Turn stage tracing on or off; `kinds` (MOE_KERNEL_* values) limits it
    to those stages."""
    if not on:
        v = 0
    elif kinds is None:
        v = 1
    else:
        v = 0
        for k in kinds:
            v |= 1 << int(k)
    return _check("moe_profile_enable", lib().moe_profile_enable(v))


def moe_profile_read(max_entries: int = 4096):
    """[(stage name, milliseconds), ...] since the last read (synchronises)."""
    kinds = (c_int32 * max_entries)()
    ms = (ctypes.c_float * max_entries)()
    n = c_int32(0)
    _check("moe_profile_read", lib().moe_profile_read(kinds, ms, max_entries, ctypes.byref(n)))
    return [(moe_kernel_name(kinds[i]), float(ms[i])) for i in range(n.value)]


def moe_kernel_name(kind: int) -> str:
    return lib().moe_kernel_name(kind).decode()
