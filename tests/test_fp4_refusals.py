"""Refusals of the 4-bit entry points, all before any CUDA call (no GPU):
the C entries with descriptors over host memory, and the argument checks of
the Python front end."""

import ctypes

import pytest
import torch

from matrix_orthogonalizing_optimizer_muon_b200 import _lib as L
from matrix_orthogonalizing_optimizer_muon_b200 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


class Mem:
    """Aligned host memory to stand for device pointers (never dereferenced)."""

    def __init__(self, n=1 << 20):
        self.buf = ctypes.create_string_buffer(n + 256)
        self.next = (ctypes.addressof(self.buf) + 255) // 256 * 256

    def take(self, n):
        p = self.next
        self.next += (n + 255) // 256 * 256
        return p


@pytest.fixture
def mem():
    return Mem()


def matrix(mem, rows, k, fmt):
    _, nd, ns = L.muon_fp4_sizes(fmt, rows, k)
    return L.muon_fp4_matrix_t(mem.take(nd), mem.take(ns), mem.take(8) if fmt == L.MUON_FP4_NV else None, rows, k, fmt, 0)


def source(mem, rows, cols, fmt, both=True):
    s = L.muon_fp4_source_t(mem.take(rows * cols * 4), cols, rows, cols, L.MUON_DT_FP32, 0)
    s.along_cols = matrix(mem, rows, cols, fmt)
    if both:
        s.along_rows = matrix(mem, cols, rows, fmt)
    else:
        s.along_rows.format = L.MUON_FP4_NONE
    return s


def test_struct_layouts():
    assert ctypes.sizeof(L.muon_fp4_matrix_t) == 48
    assert ctypes.sizeof(L.muon_fp4_source_t) == 40 + 2 * 48 + 16


def test_sizes(lib):
    assert L.muon_fp4_sizes(L.MUON_FP4_NV, 1, 1) == (16, 16, 512)
    assert L.muon_fp4_sizes(L.MUON_FP4_NV, 129, 65) == (48, 129 * 48, 2 * 2 * 512)
    assert L.muon_fp4_sizes(L.MUON_FP4_MX, 129, 129) == (80, 129 * 80, 2 * 2 * 512)
    assert L.muon_fp4_sizes(L.MUON_FP4_MX, 0, 5) == (16, 0, 0)
    assert L.muon_fp4_sizes(L.MUON_FP4_MX, 5, 0) == (0, 0, 0)
    for bad in ((2, 1, 1), (-1, 1, 1), (0, -1, 1), (0, 1, (1 << 30) + 1)):
        with pytest.raises(L.MuonError):
            L.muon_fp4_sizes(*bad)


def edit(obj, path, value):
    *head, last = path.split(".")
    for h in head:
        obj = getattr(obj, h)
    setattr(obj, last, value)


@pytest.mark.parametrize("path,value,status", [
    ("src", None, L.MUON_ERR_INVALID_ARG), ("ld", 63, L.MUON_ERR_INVALID_ARG), ("rows", -1, L.MUON_ERR_INVALID_ARG),
    ("src_dtype", 2, L.MUON_ERR_INVALID_ARG), ("reserved", 1, L.MUON_ERR_INVALID_ARG),
    ("along_cols.data", None, L.MUON_ERR_INVALID_ARG), ("along_cols.format", 7, L.MUON_ERR_INVALID_ARG),
    ("along_cols.tensor_scale", None, L.MUON_ERR_INVALID_ARG), ("along_rows.reserved", 1, L.MUON_ERR_INVALID_ARG),
    ("along_cols.format", L.MUON_FP4_MX, L.MUON_ERR_INVALID_ARG),  # the forms' formats differ
    ("along_cols.rows", 31, L.MUON_ERR_SHAPE_MISMATCH), ("along_rows.k", 64, L.MUON_ERR_SHAPE_MISMATCH),
])
def test_quantize_refusals(lib, mem, path, value, status):
    s = source(mem, 32, 64, L.MUON_FP4_NV)
    edit(s, path, value)
    assert lib.muon_fp4_quantize(ctypes.byref(s), None) == status
    plan = ctypes.c_void_p()
    arr = (L.muon_fp4_source_t * 1)(s)
    assert lib.muon_fp4_init(ctypes.byref(plan), arr, 1, -1, None) == status
    assert plan.value is None


def test_quantize_refuses_misaligned_storage_and_overlap(lib, mem):
    s = source(mem, 32, 64, L.MUON_FP4_MX)
    s.along_cols.data += 8
    assert lib.muon_fp4_quantize(ctypes.byref(s), None) == L.MUON_ERR_INVALID_ARG
    s = source(mem, 32, 64, L.MUON_FP4_MX)
    s.src += 2
    assert lib.muon_fp4_quantize(ctypes.byref(s), None) == L.MUON_ERR_INVALID_ARG
    s = source(mem, 32, 64, L.MUON_FP4_MX)
    s.along_rows.data = s.along_cols.data
    assert lib.muon_fp4_quantize(ctypes.byref(s), None) == L.MUON_ERR_ALIAS
    s = source(mem, 32, 64, L.MUON_FP4_MX)
    s.along_cols.data = s.src + 32 * 64 * 4 - 16
    assert lib.muon_fp4_quantize(ctypes.byref(s), None) == L.MUON_ERR_ALIAS
    s = source(mem, 32, 64, L.MUON_FP4_MX)
    s.along_cols.format = s.along_rows.format = L.MUON_FP4_NONE
    assert lib.muon_fp4_quantize(ctypes.byref(s), None) == L.MUON_ERR_INVALID_ARG
    assert lib.muon_fp4_quantize(None, None) == L.MUON_ERR_INVALID_ARG


def test_empty_sources_are_no_ops(lib, mem):
    for rows, cols in ((0, 64), (64, 0), (0, 0)):
        s = source(mem, rows, cols, L.MUON_FP4_NV)
        s.src = None
        assert lib.muon_fp4_quantize(ctypes.byref(s), None) == L.MUON_OK


def test_plan_refusals(lib, mem):
    plan = ctypes.c_void_p()
    a, b = source(mem, 32, 64, L.MUON_FP4_NV), source(mem, 16, 48, L.MUON_FP4_NV)

    def init(values=-1, *srcs):
        arr = (L.muon_fp4_source_t * len(srcs))(*srcs)
        return lib.muon_fp4_init(ctypes.byref(plan), arr, len(srcs), values, None)

    assert lib.muon_fp4_init(None, None, 1, -1, None) == L.MUON_ERR_INVALID_ARG
    assert lib.muon_fp4_init(ctypes.byref(plan), None, 1, -1, None) == L.MUON_ERR_INVALID_ARG
    assert init(5, a) == L.MUON_ERR_INVALID_ARG
    assert init(L.MUON_DT_BF16, a) == L.MUON_ERR_INVALID_ARG  # values wanted, nowhere to write them
    assert init(-1, a, source(mem, 16, 48, L.MUON_FP4_MX)) == L.MUON_ERR_INVALID_ARG
    assert init(-1, a, source(mem, 16, 48, L.MUON_FP4_NV, both=False)) == L.MUON_ERR_INVALID_ARG
    b.src_dtype = L.MUON_DT_BF16
    assert init(-1, a, b) == L.MUON_ERR_INVALID_ARG
    b = source(mem, 16, 48, L.MUON_FP4_NV)
    b.along_cols.scales = a.along_cols.scales
    assert init(-1, a, b) == L.MUON_ERR_ALIAS
    b = source(mem, 16, 48, L.MUON_FP4_NV)
    b.src = a.along_rows.data
    assert init(-1, a, b) == L.MUON_ERR_ALIAS
    assert plan.value is None
    assert lib.muon_fp4_run(None, None) == L.MUON_ERR_INVALID_ARG
    assert lib.muon_fp4_values(None, None) == L.MUON_ERR_INVALID_ARG
    lib.muon_fp4_destroy(None)


def test_dequantize_refusals(lib, mem):
    m = matrix(mem, 8, 40, L.MUON_FP4_MX)
    out = mem.take(8 * 40 * 4)
    call = lambda m, out, ld, dt: lib.muon_fp4_dequantize(ctypes.byref(m), out, ld, dt, None)  # noqa: E731
    assert lib.muon_fp4_dequantize(None, out, 40, 1, None) == L.MUON_ERR_INVALID_ARG
    assert call(m, None, 40, 1) == L.MUON_ERR_INVALID_ARG
    assert call(m, out, 39, 1) == L.MUON_ERR_INVALID_ARG
    assert call(m, out, 40, 2) == L.MUON_ERR_INVALID_ARG
    assert call(m, out + 2, 40, 1) == L.MUON_ERR_INVALID_ARG
    assert call(m, m.scales, 40, 0) == L.MUON_ERR_ALIAS
    assert call(matrix(mem, 0, 40, L.MUON_FP4_MX), None, 0, 1) == L.MUON_OK


def test_product_refusals(lib, mem):
    a, b = matrix(mem, 8, 40, L.MUON_FP4_NV), matrix(mem, 24, 40, L.MUON_FP4_NV)
    out = mem.take(8 * 24 * 4)

    def call(a=a, b=b, out=out, ld=24, dt=L.MUON_DT_FP32, acc=0):
        return lib.muon_fp4_product(ctypes.byref(a), ctypes.byref(b), out, ld, dt, acc, None)

    assert lib.muon_fp4_product(None, ctypes.byref(b), out, 24, 1, 0, None) == L.MUON_ERR_INVALID_ARG
    assert call(out=None) == L.MUON_ERR_INVALID_ARG
    assert call(ld=23) == L.MUON_ERR_INVALID_ARG
    assert call(dt=3) == L.MUON_ERR_INVALID_ARG
    assert call(acc=2) == L.MUON_ERR_INVALID_ARG
    assert call(dt=L.MUON_DT_BF16, acc=1) == L.MUON_ERR_INVALID_ARG
    assert call(out=out + 2) == L.MUON_ERR_INVALID_ARG
    assert call(b=matrix(mem, 24, 41, L.MUON_FP4_NV)) == L.MUON_ERR_SHAPE_MISMATCH
    assert call(b=matrix(mem, 24, 40, L.MUON_FP4_MX)) == L.MUON_ERR_SHAPE_MISMATCH
    assert call(out=b.data) == L.MUON_ERR_ALIAS
    assert call(a=matrix(mem, 0, 40, L.MUON_FP4_NV), out=None, ld=0) == L.MUON_OK


def test_rows_product_refusals(lib, mem):
    w = matrix(mem, 24, 40, L.MUON_FP4_MX)
    x, out = mem.take(33 * 40 * 2), mem.take(33 * 24 * 4)

    def call(x=x, t=3, ldx=40, w=w, out=out, ld=24, dt=L.MUON_DT_BF16):
        return lib.muon_fp4_rows_product(x, t, ldx, ctypes.byref(w), out, ld, dt, None)

    assert lib.muon_fp4_rows_product(x, 1, 40, None, out, 24, 0, None) == L.MUON_ERR_INVALID_ARG
    assert call(x=None) == L.MUON_ERR_INVALID_ARG
    assert call(x=x + 1) == L.MUON_ERR_INVALID_ARG
    assert call(t=-1) == L.MUON_ERR_INVALID_ARG
    assert call(t=L.MUON_FP4_MAX_ROWS + 1) == L.MUON_ERR_INVALID_ARG
    assert call(ldx=39) == L.MUON_ERR_INVALID_ARG
    assert call(out=None) == L.MUON_ERR_INVALID_ARG
    assert call(ld=23) == L.MUON_ERR_INVALID_ARG
    assert call(dt=4) == L.MUON_ERR_INVALID_ARG
    assert call(out=x) == L.MUON_ERR_ALIAS
    assert call(t=0, x=None, out=None, ld=0) == L.MUON_OK


def test_header_constants_match_the_binding():
    import os
    import re
    hdr = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "muon.h")).read()
    for name in ("MUON_FP4_NONE", "MUON_FP4_MX", "MUON_FP4_NV"):
        m = re.search(name + r"\s*=\s*(-?\d+)", hdr)
        assert m and int(m.group(1)) == getattr(L, name)
    m = re.search(r"#define\s+MUON_FP4_MAX_ROWS\s+(\d+)", hdr)
    assert m and int(m.group(1)) == L.MUON_FP4_MAX_ROWS


def test_front_end_refuses_host_tensors_and_bad_names():
    from matrix_orthogonalizing_optimizer_muon_b200 import fp4
    x = torch.zeros(4, 32)
    with pytest.raises(TypeError):
        fp4.fp4_quantize(x)
    with pytest.raises(TypeError):
        fp4.fp4_quantize([1.0])
    with pytest.raises(TypeError):
        fp4.Fp4Plan([x])
    with pytest.raises(ValueError):
        fp4.Fp4Plan([])
    with pytest.raises(TypeError):
        fp4.Fp4Matrix(4, 32, "mx", torch.zeros(64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(ValueError):
        fp4.Fp4Matrix(4, 32, "int4", x, x)
    with pytest.raises(TypeError):
        fp4.fp4_product(x, x)
    with pytest.raises(TypeError):
        fp4.fp4_rows_product(x, x)
    with pytest.raises(TypeError):
        fp4.fp4_linear(x, (x, x))
    with pytest.raises(TypeError):
        fp4.fp4_linear_backward((x, x), x)
