"""The training operators' argument checks (include/moe.h): every refusal
returns its documented code before anything is launched.  No GPU."""
import ctypes
import os

import pytest

from mixture_experts_layer_56_b200 import _lib as L

P = ctypes.c_void_p(0x10000)     # never dereferenced: the call is refused first
ODD = ctypes.c_void_p(0x10008)
NULL = ctypes.c_void_p(0)
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return L.lib()


def grouped(**kw):
    base = dict(rows=100, n_groups=4, n=64, k=32, dtype=L.MOE_DTYPE_BF16, flags=0)
    base.update(kw)
    return L.make_grouped_shape(**base)


GROUPED = ("moe_grouped_matmul", "moe_grouped_matmul_dx", "moe_grouped_matmul_dw")


def call(lib, fn, shape, *args):
    return getattr(lib, fn)(ctypes.byref(shape) if shape is not None else None, *args)


@pytest.mark.parametrize("fn", GROUPED)
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), L.MOE_ERR_DTYPE),
    (dict(rows=-1), L.MOE_ERR_SHAPE),
    (dict(rows=2**31 - 511), L.MOE_ERR_SHAPE),
    (dict(n_groups=0), L.MOE_ERR_SHAPE),
    (dict(n_groups=257), L.MOE_ERR_SHAPE),
    (dict(n=0), L.MOE_ERR_SHAPE),
    (dict(k=0), L.MOE_ERR_SHAPE),
    (dict(n=60), L.MOE_ERR_SHAPE),       # bf16: multiples of 8
    (dict(k=36), L.MOE_ERR_SHAPE),
    (dict(n=2**24 + 8), L.MOE_ERR_SHAPE),
    (dict(flags=4), L.MOE_ERR_SHAPE),
    (dict(flags=2), L.MOE_ERR_SHAPE),    # accumulating into bf16
    (dict(rows=2**30, n=2**20, k=8), L.MOE_ERR_SHAPE),          # tiles past int32
    (dict(n=2**20, k=2**20, rows=1), L.MOE_ERR_SHAPE),
])
def test_grouped_refuses_bad_shapes(lib, fn, kw, code):
    s = grouped(**kw)
    assert call(lib, fn, s, P, P, P, P, P, BIG, NULL) == code
    n = ctypes.c_size_t(0)
    assert lib.moe_grouped_workspace_size(ctypes.byref(s), ctypes.byref(n)) == code


@pytest.mark.parametrize("fn", GROUPED)
def test_grouped_refuses_bad_pointers(lib, fn):
    s = grouped()
    assert call(lib, fn, None, P, P, P, P, P, BIG, NULL) == L.MOE_ERR_NULLPTR
    for i in range(5):
        args = [P] * 5
        args[i] = NULL
        assert call(lib, fn, s, *args, BIG, NULL) == L.MOE_ERR_NULLPTR
        args[i] = ODD
        assert call(lib, fn, s, *args, BIG, NULL) == L.MOE_ERR_ALIGN
    need = L.moe_grouped_workspace_size(s)
    assert call(lib, fn, s, P, P, P, P, P, need - 1, NULL) == L.MOE_ERR_WORKSPACE


def test_no_rows_is_a_no_op_without_pointers(lib):
    s = grouped(rows=0)
    for fn in GROUPED[:2]:
        assert call(lib, fn, s, NULL, NULL, NULL, NULL, NULL, 0, NULL) == L.MOE_OK
    # the weight gradient of no rows is zero: it has to be written ...
    assert call(lib, GROUPED[2], s, NULL, NULL, NULL, NULL, NULL, 0, NULL) == L.MOE_ERR_NULLPTR
    assert call(lib, GROUPED[2], s, NULL, NULL, NULL, ODD, NULL, 0, NULL) == L.MOE_ERR_ALIGN
    # ... unless it is added
    s = grouped(rows=0, flags=L.MOE_GROUPED_DW_F32 | L.MOE_GROUPED_DW_ACCUMULATE)
    assert call(lib, GROUPED[2], s, NULL, NULL, NULL, NULL, NULL, 0, NULL) == L.MOE_OK
    sw = L.make_swiglu_shape(0, 64)
    assert call(lib, "moe_swiglu", sw, NULL, NULL, NULL) == L.MOE_OK
    assert call(lib, "moe_swiglu_backward", sw, NULL, NULL, NULL, NULL) == L.MOE_OK
    nm = L.make_norm_shape(0, 64)
    assert call(lib, "moe_layer_norm", nm, *[NULL] * 6, NULL) == L.MOE_OK
    om = L.make_ortho_shape(0, 64, 64)
    assert call(lib, "moe_orthogonalize", om, None, NULL, NULL, NULL, 0, NULL) == L.MOE_OK


def test_fp32_takes_any_width(lib):
    assert L.moe_grouped_workspace_size(grouped(n=7, k=1, dtype=L.MOE_DTYPE_F32)) >= 256


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), L.MOE_ERR_DTYPE), (dict(rows=-1), L.MOE_ERR_SHAPE),
    (dict(rows=2**31), L.MOE_ERR_SHAPE), (dict(inter=0), L.MOE_ERR_SHAPE),
    (dict(inter=96), L.MOE_ERR_SHAPE), (dict(inter=2**24 + 64), L.MOE_ERR_SHAPE),
])
def test_swiglu_refusals(lib, kw, code):
    base = dict(rows=4, inter=64, dtype=L.MOE_DTYPE_BF16)
    base.update(kw)
    s = L.make_swiglu_shape(**base)
    assert call(lib, "moe_swiglu", s, P, P, NULL) == code
    assert call(lib, "moe_swiglu_backward", s, P, P, P, NULL) == code


def test_swiglu_refuses_bad_pointers(lib):
    s = L.make_swiglu_shape(4, 64)
    assert call(lib, "moe_swiglu", None, P, P, NULL) == L.MOE_ERR_NULLPTR
    for bad, code in ((NULL, L.MOE_ERR_NULLPTR), (ODD, L.MOE_ERR_ALIGN)):
        for i in range(2):
            a = [P, P]
            a[i] = bad
            assert call(lib, "moe_swiglu", s, *a, NULL) == code
        for i in range(3):
            a = [P, P, P]
            a[i] = bad
            assert call(lib, "moe_swiglu_backward", s, *a, NULL) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=-1), L.MOE_ERR_DTYPE), (dict(T=-1), L.MOE_ERR_SHAPE),
    (dict(T=2**31), L.MOE_ERR_SHAPE), (dict(d=0), L.MOE_ERR_SHAPE),
    (dict(d=2**24 + 1), L.MOE_ERR_SHAPE), (dict(eps=-1e-5), L.MOE_ERR_SHAPE),
    (dict(eps=float("nan")), L.MOE_ERR_SHAPE), (dict(eps=float("inf")), L.MOE_ERR_SHAPE),
])
def test_norm_refuses_bad_shapes(lib, kw, code):
    base = dict(T=4, d=64, dtype=L.MOE_DTYPE_BF16, eps=1e-5)
    base.update(kw)
    s = L.make_norm_shape(**base)
    assert call(lib, "moe_layer_norm", s, *[P] * 6, NULL) == code
    assert call(lib, "moe_layer_norm_backward", s, *[P] * 9, BIG, NULL) == code
    n = ctypes.c_size_t(0)
    assert lib.moe_layer_norm_workspace_size(ctypes.byref(s), ctypes.byref(n)) == code


def test_norm_refuses_bad_pointers(lib):
    s = L.make_norm_shape(4, 64)
    assert call(lib, "moe_layer_norm", None, *[P] * 6, NULL) == L.MOE_ERR_NULLPTR
    for i in range(6):      # x gamma beta y mean rstd
        a = [P] * 6
        a[i] = ODD
        assert call(lib, "moe_layer_norm", s, *a, NULL) == L.MOE_ERR_ALIGN
        if i in (0, 1, 3):
            a[i] = NULL
            assert call(lib, "moe_layer_norm", s, *a, NULL) == L.MOE_ERR_NULLPTR
    need = L.moe_layer_norm_workspace_size(s)
    for i in range(9):      # dy x gamma mean rstd dx dgamma dbeta ws
        a = [P] * 9
        a[i] = ODD
        assert call(lib, "moe_layer_norm_backward", s, *a, need, NULL) == L.MOE_ERR_ALIGN
        if i != 7:
            a[i] = NULL
            assert call(lib, "moe_layer_norm_backward", s, *a, need, NULL) == L.MOE_ERR_NULLPTR
    assert call(lib, "moe_layer_norm_backward", s, *[P] * 9, need - 1, NULL) == L.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), L.MOE_ERR_DTYPE), (dict(n_mats=-1), L.MOE_ERR_SHAPE),
    (dict(n_mats=65536), L.MOE_ERR_SHAPE), (dict(rows=0), L.MOE_ERR_SHAPE),
    (dict(cols=0), L.MOE_ERR_SHAPE), (dict(rows=65537), L.MOE_ERR_SHAPE),
    (dict(cols=65537), L.MOE_ERR_SHAPE), (dict(steps=0), L.MOE_ERR_SHAPE),
    (dict(steps=17), L.MOE_ERR_SHAPE),
    (dict(n_mats=65535, rows=65536, cols=65536), L.MOE_ERR_SHAPE),
])
def test_orthogonalize_refuses_bad_shapes(lib, kw, code):
    base = dict(n_mats=1, rows=16, cols=32, steps=5, dtype=L.MOE_DTYPE_F32)
    base.update(kw)
    s = L.make_ortho_shape(**base)
    assert call(lib, "moe_orthogonalize", s, None, P, P, P, BIG, NULL) == code
    n = ctypes.c_size_t(0)
    assert lib.moe_orthogonalize_workspace_size(ctypes.byref(s), ctypes.byref(n)) == code


def test_orthogonalize_refuses_bad_pointers(lib):
    s = L.make_ortho_shape(2, 16, 32)
    need = L.moe_orthogonalize_workspace_size(s)
    for i in range(3):
        a = [P] * 3
        a[i] = NULL
        assert call(lib, "moe_orthogonalize", s, None, *a, need, NULL) == L.MOE_ERR_NULLPTR
        a[i] = ODD
        assert call(lib, "moe_orthogonalize", s, None, *a, need, NULL) == L.MOE_ERR_ALIGN
    assert call(lib, "moe_orthogonalize", s, None, P, P, P, need - 1, NULL) == L.MOE_ERR_WORKSPACE
    with pytest.raises(ValueError):
        L.moe_orthogonalize(s, 0x10000, 0x10000, 0x10000, ws_bytes=need, coef=[1.0, 2.0], stream=0)


def test_workspaces_grow_with_their_shapes(lib):
    sizes = [L.moe_orthogonalize_workspace_size(L.make_ortho_shape(n, 148, 180)) for n in (1, 2, 9)]
    assert sizes[0] < sizes[1] < sizes[2] and all(x % 256 == 0 for x in sizes)
    # matrices that stay on chip need the status word alone
    assert [L.moe_orthogonalize_workspace_size(L.make_ortho_shape(n, *rc)) for n in (1, 9)
            for rc in ((48, 80), (2048, 128))] == [256] * 4
    assert L.moe_layer_norm_workspace_size(L.make_norm_shape(0, 64)) == 0
    assert (L.moe_layer_norm_workspace_size(L.make_norm_shape(1, 64))
            < L.moe_layer_norm_workspace_size(L.make_norm_shape(4096, 64)))


def test_nothing_was_launched(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("other tests launch kernels here")
    assert L.moe_launch_count() == 0
