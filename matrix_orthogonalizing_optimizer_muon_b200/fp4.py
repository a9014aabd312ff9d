"""Microscaled 4-bit matrices over torch tensors: quantisation, products, and a
linear layer that trains with 4-bit products.

A 4-bit matrix [rows, k] holds e2m1 codes and one scale a block of
consecutive k: fmt "mx" (blocks of 32, power-of-two scales) or "nv" (blocks
of 16, e4m3 scales times one power of two per matrix); include/muon.h states
the rounding and the storage.

    q = fp4_quantize(x)                      # [R, C] -> blocks along C
    qt = fp4_quantize(x, along="rows")       # blocks along R: the transpose [C, R]
    y = fp4_product(q, wq)                   # q @ wq.T, 4-bit tensor-core products
    y = fp4_rows_product(tokens, wq)         # a few bf16 rows, unquantised

The weights' 4-bit copies are made, and refreshed after an optimizer step, by
one plan:

    plan = Fp4Plan(weights, along="both")    # quantises them as they are now
    opt = HybridStep(..., fp4=plan)          # or plan.run() after any step
    y, kept = fp4_linear(x, plan.matrices[i])
    dx, dw = fp4_linear_backward(kept, dy)   # dw is the gradient that the step takes

Work is enqueued on `stream`, or the current stream of the operands' device;
tensors that a call allocates belong to that stream.  An operand made on
another stream has to be ready before, as for any torch call, and must not be
freed there before the call's work is done (torch's record_stream).  Nothing
here builds an autograd graph, and nothing but a plan's set-up and the status
read synchronises.
"""

from __future__ import annotations

import ctypes
from contextlib import nullcontext

import torch

from . import _lib as L
from .api import _GDT

_FMT = {"mx": L.MUON_FP4_MX, "nv": L.MUON_FP4_NV}
_BLOCK = {"mx": 32, "nv": 16}
MAX_ROWS = L.MUON_FP4_MAX_ROWS
_MAX_DIM = 1 << 30


_NOTHING = nullcontext()


def _on(device, stream):
    """A context with the operands' device current and `stream`, if given, its current stream."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the operands on {device}")
        return torch.cuda.stream(stream)
    if torch._C._cuda_getDevice() != device.index:
        return torch.cuda.device(device)
    return _NOTHING


def _current(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def _sizes(fmt: str, rows: int, k: int):
    """(bytes of the codes, bytes of the scales), as muon_fp4_sizes gives them."""
    return rows * (-(-k // 32) * 16), -(-rows // 128) * -(-k // (4 * _BLOCK[fmt])) * 512


def _matrix_arg(t, name: str, dtypes=(torch.bfloat16, torch.float32)) -> int:
    """Check a 2-D row-major tensor (any row pitch); returns the pitch."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows (for a transposed view, pass the matrix and the other "
                         "`along`)")
    ld = t.stride(0) if rows > 1 else cols
    if ld < cols or (rows > 1 and ld < 1):
        raise ValueError(f"the rows of {name} overlap (stride {t.stride(0)})")
    return ld


def _check_fmt(fmt: str) -> None:
    if fmt not in _FMT:
        raise ValueError(f"fmt must be one of {sorted(_FMT)}, got {fmt!r}")


def _part(t, name: str, dtype, n: int) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} elements, got {tuple(t.shape)}")


class Fp4Matrix:
    """A 4-bit matrix [rows, k] on the device: codes `data` (uint8), `scales`
    (uint8) and, for "nv", `tensor_scale` (fp32: g and the largest magnitude),
    laid out as include/muon.h states."""

    def __init__(self, rows: int, k: int, fmt: str, data: torch.Tensor, scales: torch.Tensor,
                 tensor_scale: torch.Tensor | None = None):
        _check_fmt(fmt)
        rows, k = int(rows), int(k)
        if rows < 0 or k < 0 or rows > _MAX_DIM or k > _MAX_DIM:
            raise ValueError(f"a 4-bit matrix has 0 to 2^30 rows and columns, not {rows} x {k}")
        data_bytes, scale_bytes = _sizes(fmt, rows, k)
        _part(data, "data", torch.uint8, data_bytes)
        _part(scales, "scales", torch.uint8, scale_bytes)
        device = data.device
        if fmt == "nv":
            _part(tensor_scale, "tensor_scale", torch.float32, 2)
        if scales.device != device or (fmt == "nv" and tensor_scale.device != device):
            raise ValueError("data, scales and tensor_scale are on different devices")
        self._set(rows, k, fmt, device, data.data_ptr(), scales.data_ptr(),
                  tensor_scale.data_ptr() if fmt == "nv" else None)
        self._parts = data, scales, tensor_scale if fmt == "nv" else None

    def _set(self, rows, k, fmt, device, data_ptr, scales_ptr, ts_ptr):
        self.rows, self.k, self.fmt, self.device = rows, k, fmt, device
        self._desc = L.muon_fp4_matrix_t(data_ptr, scales_ptr, ts_ptr, rows, k, _FMT[fmt], 0)

    @classmethod
    def empty(cls, rows: int, k: int, fmt: str = "nv", device=None) -> "Fp4Matrix":
        """Uninitialised storage in one allocation."""
        _check_fmt(fmt)
        return cls._alloc([(rows, k)], fmt, device if device is not None else "cuda")[0]

    @classmethod
    def _alloc(cls, shapes, fmt, device):
        """Uninitialised matrices of these shapes in one allocation."""
        plan, end = [], 0
        for rows, k in shapes:
            if rows < 0 or k < 0 or rows > _MAX_DIM or k > _MAX_DIM:
                raise ValueError(f"a 4-bit matrix has 0 to 2^30 rows and columns, not {rows} x {k}")
            nd, ns = _sizes(fmt, rows, k)
            off = end + -(-nd // 256) * 256
            plan.append((rows, k, end, nd, off, ns))
            end = off + ns + 256  # the tensor scale, and the next matrix on a 256-byte boundary
        buf = torch.empty(end, dtype=torch.uint8, device=device)
        at, dev, nv, out = buf.data_ptr(), buf.device, fmt == "nv", []
        for rows, k, start, nd, off, ns in plan:
            m = cls.__new__(cls)
            m._set(rows, k, fmt, dev, at + start, at + off, at + off + ns if nv else None)
            m._parts, m._buf = None, (buf, start, nd, off, ns)
            out.append(m)
        return out

    def _views(self):
        """(codes, scales, tensor scale) as tensors; cut from the allocation when first asked for."""
        if self._parts is None:
            buf, start, nd, off, ns = self._buf
            self._parts = (buf[start:start + nd], buf[off:off + ns],
                           buf[off + ns:off + ns + 8].view(torch.float32) if self.fmt == "nv" else None)
        return self._parts

    @property
    def data(self) -> torch.Tensor:
        return self._views()[0]

    @property
    def scales(self) -> torch.Tensor:
        return self._views()[1]

    @property
    def tensor_scale(self) -> torch.Tensor | None:
        return self._views()[2]

    @property
    def shape(self):
        return self.rows, self.k

    def dequantize(self, dtype=torch.bfloat16, *, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The values [rows, k] in bf16 or fp32 (or into `out`)."""
        with _on(self.device, stream):
            out, ld = _out(out, (self.rows, self.k), dtype, self.device)
            L.muon_fp4_dequantize(self._desc, out.data_ptr(), ld, _GDT[out.dtype], _current(self.device))
        return out


def _out(out, shape, dtype, device):
    """(the output, its row pitch): a new tensor of `dtype`, or a given one that fits."""
    if out is None:
        if dtype not in _GDT:
            raise TypeError(f"output dtype {dtype}: bf16 or fp32")
        return torch.empty(shape, dtype=dtype, device=device), shape[1]
    ld = _matrix_arg(out, "out")
    if out.shape != shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {shape}")
    if out.device != device:
        raise ValueError(f"out is on {out.device}, the operands on {device}")
    return out, ld


def _ways(along: str):
    if along not in ("cols", "rows", "both"):
        raise ValueError(f"along must be 'cols', 'rows' or 'both', got {along!r}")
    return along != "rows", along != "cols"


def _source(x, fmt, along, out):
    """(source descriptor, the 4-bit matrices it is written to, in the order cols, rows)."""
    ld = _matrix_arg(x, "x")
    _check_fmt(fmt)
    want_c, want_r = _ways(along)
    rows, cols = x.shape
    shapes = [(rows, cols)] * want_c + [(cols, rows)] * want_r
    if out is None:
        out = Fp4Matrix._alloc(shapes, fmt, x.device)
    else:
        out = list(out) if along == "both" else [out]
        if len(out) != len(shapes) or not all(isinstance(m, Fp4Matrix) for m in out):
            raise TypeError("out must be an Fp4Matrix, or the pair (cols, rows) for along='both'")
        for m, s in zip(out, shapes):
            if m.shape != s or m.fmt != fmt:
                raise ValueError(f"out is a {m.fmt} matrix {m.shape}, expected {fmt} {s}")
            if m.device != x.device:
                raise ValueError(f"out is on {m.device}, x on {x.device}")
    src = L.muon_fp4_source_t(x.data_ptr(), ld, rows, cols, _GDT[x.dtype], 0)
    src.along_cols.format = src.along_rows.format = L.MUON_FP4_NONE
    if want_c:
        src.along_cols = out[0]._desc
    if want_r:
        src.along_rows = out[-1]._desc
    return src, out


def fp4_quantize(x: torch.Tensor, *, fmt: str = "nv", along: str = "cols", out=None, stream=None):
    """Quantise x [R, C] (bf16 or fp32, any row pitch): along="cols" gives an
    Fp4Matrix [R, C] with blocks along C, "rows" its transpose [C, R] with
    blocks along R, "both" the pair of them from one read."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    with _on(x.device, stream):
        src, out = _source(x, fmt, along, out)
        L.muon_fp4_quantize(src, _current(x.device))
    return tuple(out) if along == "both" else out[0]


class Fp4Plan:
    """Quantises a fixed list of tensors [R, C] (one dtype) in one pass each
    run: the 4-bit copies of a model's weights.  `matrices[i]` is the
    Fp4Matrix of tensors[i], or the pair (cols, rows) for along="both"; the
    set-up runs the plan once, so they hold the tensors as they are then, and
    waits for that.  With `values` (bf16 or fp32) the plan also holds dense
    tensors for ``dequantize``."""

    def __init__(self, tensors, *, fmt: str = "nv", along: str = "cols", values: torch.dtype | None = None, stream=None):
        tensors = list(tensors)
        if not tensors:
            raise ValueError("a 4-bit plan needs at least one tensor")
        for i, t in enumerate(tensors):
            _matrix_arg(t, f"tensors[{i}]")
            if t.dtype != tensors[0].dtype or t.device != tensors[0].device:
                raise ValueError("all tensors of a plan share a dtype and a device")
        if values is not None and values not in _GDT:
            raise TypeError(f"values dtype {values}: bf16 or fp32")
        self.device = tensors[0].device
        self._keep = tensors  # the plan holds raw pointers: keep the tensors alive
        self._plan = None
        with _on(self.device, stream):
            srcs = (L.muon_fp4_source_t * len(tensors))()
            self.matrices, self._values = [], [[] for _ in range(2 if along == "both" else 1)]
            for i, t in enumerate(tensors):
                src, out = _source(t, fmt, along, None)
                self.matrices.append(tuple(out) if along == "both" else out[0])
                if values is not None:
                    dense = [torch.empty(m.shape, dtype=values, device=self.device) for m in out]
                    for v, d in zip(self._values, dense):
                        v.append(d)
                    src.values_cols = dense[0].data_ptr() if along != "rows" else None
                    src.values_rows = dense[-1].data_ptr() if along != "cols" else None
                srcs[i] = src
            self._plan = L.muon_fp4_init(srcs, len(tensors), -1 if values is None else _GDT[values],
                                         _current(self.device))
            L.muon_fp4_run(self._plan, _current(self.device))
            torch.cuda.current_stream(self.device).synchronize()  # a next run, on any stream, must not overlap

    def run(self, stream=None) -> None:
        """Quantise every tensor as it is now."""
        with _on(self.device, stream):
            L.muon_fp4_run(self._plan, _current(self.device))

    def dequantize(self, stream=None):
        """The values of every 4-bit matrix, into the plan's dense tensors:
        one list per form, in the order (cols, rows)."""
        with _on(self.device, stream):
            L.muon_fp4_values(self._plan, _current(self.device))
        return [list(v) for v in self._values]

    def close(self) -> None:
        if getattr(self, "_plan", None):
            L.muon_fp4_destroy(self._plan)
            self._plan = None
            self._keep = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _operand(m, name: str) -> None:
    if not isinstance(m, Fp4Matrix):
        raise TypeError(f"{name} must be an Fp4Matrix")


def fp4_product(a: Fp4Matrix, b: Fp4Matrix, *, out: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                accumulate: bool = False, stream=None) -> torch.Tensor:
    """a @ b.T of two 4-bit matrices [M, k] and [N, k] of one format, with
    fp32 sums; accumulate=True adds it to `out` (fp32)."""
    _operand(a, "a")
    _operand(b, "b")
    if a.k != b.k or a.fmt != b.fmt:
        raise ValueError(f"a is {a.fmt} {a.shape}, b is {b.fmt} {b.shape}: one format and one k are needed")
    if a.device != b.device:
        raise ValueError(f"a is on {a.device}, b on {b.device}")
    if accumulate and (out is None or out.dtype != torch.float32):
        raise ValueError("accumulate adds to an fp32 `out`")
    with _on(a.device, stream):
        out, ld = _out(out, (a.rows, b.rows), out_dtype, a.device)
        L.muon_fp4_product(a._desc, b._desc, out.data_ptr(), ld, _GDT[out.dtype], 1 if accumulate else 0,
                           _current(a.device))
    return out


def fp4_rows_product(x: torch.Tensor, w: Fp4Matrix, *, out: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                     stream=None) -> torch.Tensor:
    """x @ w.T for a few bf16 rows x [t, k], t <= 32, and a 4-bit matrix w
    [N, k]; a row's result does not depend on the other rows.  For more rows,
    quantise x and use ``fp4_product``."""
    _operand(w, "w")
    ldx = _matrix_arg(x, "x", (torch.bfloat16,))
    if x.device != w.device:
        raise ValueError(f"x is on {x.device}, w on {w.device}")
    if x.shape[1] != w.k:
        raise ValueError(f"x has {x.shape[1]} columns, w has k = {w.k}")
    if x.shape[0] > MAX_ROWS:
        raise ValueError(f"x has {x.shape[0]} rows, at most {MAX_ROWS} are taken: quantise it and use fp4_product")
    with _on(w.device, stream):
        out, ld = _out(out, (x.shape[0], w.rows), out_dtype, w.device)
        L.muon_fp4_rows_product(x.data_ptr(), x.shape[0], ldx, w._desc, out.data_ptr(), ld, _GDT[out.dtype],
                                _current(w.device))
    return out


class Fp4Kept:
    """What a linear layer's forward pass keeps for its backward pass: x along
    the tokens and w along the outputs, both in 4 bits."""

    def __init__(self, xt: Fp4Matrix, w: Fp4Matrix):
        self.xt, self.w = xt, w


def _both(x, name: str, fmt: str, device, st: int):
    """Both forms (along cols, along rows) of a matrix, on the current device and stream."""
    ld = _matrix_arg(x, name)
    rows, cols = x.shape
    c, r = Fp4Matrix._alloc(((rows, cols), (cols, rows)), fmt, device)
    L.muon_fp4_quantize(L.muon_fp4_source_t(x.data_ptr(), ld, rows, cols, _GDT[x.dtype], 0, c._desc, r._desc), st)
    return c, r


def _times(a: Fp4Matrix, b: Fp4Matrix, out, dtype, accumulate: bool, st: int):
    """fp4_product of matrices that are known to fit, on the current device and stream."""
    out, ld = _out(out, (a.rows, b.rows), dtype, a.device)
    L.muon_fp4_product(a._desc, b._desc, out.data_ptr(), ld, _GDT[out.dtype], 1 if accumulate else 0, st)
    return out


def fp4_linear(x: torch.Tensor, w, *, fmt: str | None = None, out_dtype=torch.bfloat16, stream=None):
    """y = Q(x) Q(w) for x [T, K] and a weight w [K, N], Q the rounding to 4
    bits in blocks along the summed dimension.  w is a tensor, or the pair
    (along cols, along rows) that fp4_quantize or an Fp4Plan made of it with
    along="both".  Returns (y [T, N], what fp4_linear_backward needs).

    x and w are taken as values: no autograd graph is built, whether they
    require gradients or not (fp4_linear_backward gives them).  What is kept
    refers to a given pair itself, so the backward pass belongs before the
    plan of that pair runs again."""
    _matrix_arg(x, "x")
    device = x.device
    if isinstance(w, torch.Tensor):
        fmt = fmt or "nv"
        _check_fmt(fmt)
        _matrix_arg(w, "w")
        shape, w_device = w.shape, w.device
    else:
        if not (isinstance(w, (tuple, list)) and len(w) == 2 and all(isinstance(m, Fp4Matrix) for m in w)):
            raise TypeError("w must be a tensor or the pair (along cols, along rows) of its 4-bit forms")
        w_cols, w_rows = w
        if w_cols.shape != w_rows.shape[::-1] or w_cols.fmt != w_rows.fmt or w_cols.device != w_rows.device:
            raise ValueError(f"the forms of w do not belong together: {w_cols.fmt} {w_cols.shape}, "
                             f"{w_rows.fmt} {w_rows.shape}")
        if fmt is not None and fmt != w_cols.fmt:
            raise ValueError(f"w is in format {w_cols.fmt}, not {fmt}")
        fmt, shape, w_device = w_cols.fmt, w_cols.shape, w_cols.device
    if x.shape[1] != shape[0]:
        raise ValueError(f"x has {x.shape[1]} columns, w has {shape[0]} rows")
    if w_device != device:
        raise ValueError(f"x is on {device}, w on {w_device}")
    if out_dtype not in _GDT:
        raise TypeError(f"out_dtype {out_dtype}: bf16 or fp32")
    with _on(device, stream):
        st = _current(device)
        if isinstance(w, torch.Tensor):
            w_cols, w_rows = _both(w, "w", fmt, device, st)
        xq, xt = _both(x, "x", fmt, device, st)
        return _times(xq, w_rows, None, out_dtype, False, st), Fp4Kept(xt, w_cols)


def fp4_linear_backward(kept: Fp4Kept, dy: torch.Tensor, *, dw: torch.Tensor | None = None, accumulate: bool = False,
                        dx_dtype=torch.bfloat16, stream=None):
    """(dx, dw) of a linear layer from dy [T, N]: dx = Q(dy) Q(w)^T and
    dw = Q(x)^T Q(dy), every operand rounded to 4 bits in blocks along its
    product's summed dimension, the roundings passed through unchanged.  dw is
    fp32 [K, N]; a given one is written (bf16 or fp32), or with
    accumulate=True added to (fp32), which gathers several micro-batches."""
    if not isinstance(kept, Fp4Kept):
        raise TypeError("kept must come from fp4_linear")
    tokens, n, device, fmt = kept.xt.k, kept.w.k, kept.w.device, kept.w.fmt
    _matrix_arg(dy, "dy")
    if tuple(dy.shape) != (tokens, n):
        raise ValueError(f"dy has shape {tuple(dy.shape)}, expected {(tokens, n)}")
    if dy.device != device:
        raise ValueError(f"dy is on {dy.device}, the layer on {device}")
    if accumulate and (dw is None or dw.dtype != torch.float32):
        raise ValueError("accumulate adds to a given fp32 dw")
    if dw is not None:
        _out(dw, (kept.xt.rows, n), None, device)  # refused before anything is enqueued
    if dx_dtype not in _GDT:
        raise TypeError(f"dx_dtype {dx_dtype}: bf16 or fp32")
    with _on(device, stream):
        st = _current(device)
        dyq, dyt = _both(dy, "dy", fmt, device, st)
        dx = _times(dyq, kept.w, None, dx_dtype, False, st)
        return dx, _times(kept.xt, dyt, dw, torch.float32, accumulate, st)


def fp4_status(stream=None) -> int:
    """Synchronising read-and-clear of the device status of the 4-bit products
    (MUON_OK, or MUON_ERR_TIMEOUT after a device-side wait gave up)."""
    device = stream.device if stream is not None else torch.device("cuda", torch.cuda.current_device())
    with _on(device, stream):
        return L.muon_fp4_get_status(_current(device))
