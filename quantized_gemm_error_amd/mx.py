"""Binding of libspear's microscaled matrices, norm and linear (include/spear_mx.h), same names as
the C ABI.

Argument marshalling and checks only, as in spear.py: every step runs in the library's HIP
kernels, and there is no fallback.  A SpearMX handle checks its tensors once and keeps the C
struct; a program makes its weights' once.
"""

from __future__ import annotations

import ctypes

from . import spear
from .attn import _INT32_MAX, _fits, _gpu, _meet, _On, _span
from .spear import SPEAR_ERR_INVALID_ARGUMENT, SpearError, _check, _require

SPEAR_MXFP4, SPEAR_MXFP8 = 0, 1
SPEAR_F32 = 2

# Every function the header declares, for the export check.
EXPORTED = (
    "spear_mx_code_bytes", "spear_mx_scale_bytes", "spear_mx_quantize", "spear_mx_dequantize",
    "spear_rms_norm", "spear_mx_workspace_bytes", "spear_mx_linear",
)

_P, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_FORMATS = {"fp4": SPEAR_MXFP4, "fp8": SPEAR_MXFP8, SPEAR_MXFP4: SPEAR_MXFP4, SPEAR_MXFP8: SPEAR_MXFP8}


class SpearMXC(ctypes.Structure):
    _fields_ = [("format", _i32), ("rows", _i32), ("cols", _i32), ("codes", _P), ("scales", _P)]


class SpearNormArgsC(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("rows", _i32), ("hidden", _i32),
                ("x", _P), ("residual", _P), ("weight", _P),
                ("x_stride", _i64), ("residual_stride", _i64),
                ("residual_out", _P), ("out", _P),
                ("residual_out_stride", _i64), ("out_stride", _i64),
                ("out_mx", _P), ("eps", ctypes.c_double)]


class SpearMXLinearArgsC(ctypes.Structure):
    _fields_ = [("w", _P), ("x_mx", _P), ("x", _P), ("x_dtype", _i32), ("x_format", _i32),
                ("n_tokens", _i32), ("x_stride", _i64), ("y", _P), ("y_dtype", _i32), ("y_stride", _i64)]


_bound = None


def load_library():
    """libspear.so with this header's functions declared (raises if it has not been built)."""
    global _bound
    if _bound is not None:
        return _bound
    lib = spear.load_library()
    for name, args in (("spear_mx_code_bytes", [_i32, _i32, _i32]),
                       ("spear_mx_scale_bytes", [_i32, _i32, _i32]),
                       ("spear_mx_workspace_bytes", [_P, _i32]),
                       ("spear_mx_quantize", [_P, _i32, _i64, _P, _P]),
                       ("spear_mx_dequantize", [_P, _P, _i32, _i64, _P]),
                       ("spear_rms_norm", [_P, _P]),
                       ("spear_mx_linear", [_P, _P, _sz, _P])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = _sz if name.endswith("bytes") else _i32
    _bound = lib
    return lib


def _lib():
    return _bound if _bound is not None else load_library()


def _format(fmt) -> int:
    try:
        return _FORMATS[fmt]
    except (KeyError, TypeError):
        raise ValueError(f"format {fmt!r} is not 'fp4' or 'fp8'") from None


_codes = None


def _dtype_code(dtype, name: str, f32: bool = True) -> int:
    global _codes
    if _codes is None:
        import torch
        _codes = {torch.float16: spear.SPEAR_F16, torch.bfloat16: spear.SPEAR_BF16, torch.float32: SPEAR_F32}
    code = _codes.get(dtype)
    if code is None or (code == SPEAR_F32 and not f32):
        raise TypeError(f"{name} must be float16{',' if f32 else ' or'} bfloat16"
                        f"{' or float32' if f32 else ''}, got {dtype}")
    return code


def _matrix(t, name: str, f32: bool = True):
    """t is [rows][cols] with contiguous columns -> its type's code, sizes and row stride."""
    _require(t.dim() == 2, f"{name} must be [rows][cols], got {t.dim()}-D")
    rows, cols = t.shape
    if rows > _INT32_MAX or cols > _INT32_MAX:
        _fits(rows, f"rows of {name}"), _fits(cols, f"columns of {name}")
    stride, inner = t.stride()
    if cols > 1 and inner != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return _dtype_code(t.dtype, name, f32), rows, cols, stride


def _as(t, name: str, dtype, device, shape):
    """t has this dtype, device and shape, contiguous columns -> its row stride."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dim() == 1:
        _require(t.numel() < 2 or t.stride(0) == 1, f"{name} must be contiguous")
        return 0
    if shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0)


def _same_rows(a, b) -> bool:
    return a.data_ptr() == b.data_ptr() and (a.shape[0] < 2 or a.stride(0) == b.stride(0))


class SpearMX:
    """A microscaled matrix (spear_mx_t): codes and scales as uint8 device tensors in the header's
    order, format "fp4" or "fp8"."""

    def __init__(self, codes, scales, rows: int, cols: int, fmt):
        import torch
        fmt = _format(fmt)
        need = _mx_bytes(fmt, rows, cols)
        for t, name, n in ((codes, "codes", need[0]), (scales, "scales", need[1])):
            _require(t.dtype == torch.uint8, f"{name} must be uint8", TypeError)
            _require(t.dim() == 1 and t.is_contiguous() and t.numel() == n,
                     f"{name} must be contiguous, of {n} bytes")
        _require(codes.device == scales.device, f"codes are on {codes.device}, scales on {scales.device}")
        self._parts, self.device = (codes, scales), codes.device
        self._set(fmt, rows, cols, codes.data_ptr(), scales.data_ptr())

    def _set(self, fmt, rows, cols, codes_at, scales_at):
        self.rows, self.cols, self.format, self.shape = rows, cols, fmt, (rows, cols)
        self.c = SpearMXC(fmt, rows, cols, codes_at, scales_at)
        self.at = ctypes.addressof(self.c)

    @classmethod
    def empty(cls, rows: int, cols: int, fmt, device="cuda") -> "SpearMX":
        """A matrix whose values are not set."""
        import torch
        fmt = _format(fmt)
        codes, scales = _mx_bytes(fmt, rows, cols)
        # one allocation: a device's allocations start at 512-byte places, and codes is a multiple of 1024
        both = torch.empty(codes + scales, dtype=torch.uint8, device=device)
        self = cls.__new__(cls)
        self._both, self._parts, self.device = both, None, both.device
        at = both.data_ptr()
        self._set(fmt, rows, cols, at, at + codes)
        return self

    def _tensors(self):
        if self._parts is None:
            n = _mx_bytes(self.format, self.rows, self.cols)[0]
            self._parts = self._both[:n], self._both[n:]
        return self._parts

    @property
    def codes(self):
        return self._tensors()[0]

    @property
    def scales(self):
        return self._tensors()[1]

    @property
    def spans(self):
        return tuple(_span(t) for t in self._tensors())


def _mx_bytes(fmt: int, rows: int, cols: int):
    """spear_mx_code_bytes and spear_mx_scale_bytes."""
    if not (0 <= rows <= 1 << 24 and 1 <= cols <= 1 << 20):
        _fits(rows, "rows"), _fits(cols, "cols")
        raise SpearError(SPEAR_ERR_INVALID_ARGUMENT, f"invalid sizes {rows} x {cols}")
    blocks = (rows + 15) >> 4
    return blocks * ((cols + 127) >> 7) * (2048 if fmt else 1024), blocks * ((cols + 511) >> 9) * 256


def _meets(mx: SpearMX, span) -> bool:
    return _meet(mx.spans[0], span) or _meet(mx.spans[1], span)


def spear_mx_quantize(x, fmt=None, out: SpearMX = None, stream=None) -> SpearMX:
    """x [rows][cols] (float16, bfloat16 or float32) as a microscaled matrix of format fmt (None:
    out's, or "fp4")."""
    code, rows, cols, stride = _matrix(x, "x")
    device = x.device
    if out is not None:
        _require(out.device == device, f"out is on {out.device}, x on {device}")
        _require(out.shape == (rows, cols), f"out is {out.shape}, x {(rows, cols)}")
        _require(fmt is None or _format(fmt) == out.format, "out has another format")
        _require(not _meets(out, _span(x)), "out must not overlap x")
    _gpu(device)
    on = _On(device, stream)
    if out is None:
        out = SpearMX.empty(rows, cols, "fp4" if fmt is None else fmt, device)
        if on.given:
            on.made(out._both)
    with on as ptr:
        status = _lib().spear_mx_quantize(x.data_ptr(), code, stride, out.at, ptr)
    if status:
        _check(status)
    return out


def spear_mx_dequantize(x: SpearMX, dtype=None, out=None, stream=None):
    """The values of x [rows][cols] as dtype (out's, or float32)."""
    import torch
    if dtype is None:
        dtype = torch.float32 if out is None else out.dtype
    code = _dtype_code(dtype, "dtype")
    stride = x.cols
    if out is not None:
        stride = _as(out, "out", dtype, x.device, x.shape)
        _require(not _meets(x, _span(out)), "out must not overlap x")
    _gpu(x.device)
    on = _On(x.device, stream)
    if out is None:
        out = torch.empty(x.shape, dtype=dtype, device=x.device)
        if on.given:
            on.made(out)
    with on as ptr:
        status = _lib().spear_mx_dequantize(x.at, out.data_ptr(), code, stride, ptr)
    if status:
        _check(status)
    return out


def _norm_overlaps(x, weight, residual, residual_out, out, mx):
    """An output may lie where x or the residual lies if it is the same rows, and nowhere else."""
    ins = [(n, t) for n, t in (("x", x), ("weight", weight), ("residual", residual)) if t is not None]
    outs = [] if residual_out is None else [("residual_out", residual_out)]
    if mx and out is not None:
        for name, t in ins + outs:
            _require(not _meets(out, _span(t)), f"out must not overlap {name}")
    elif out is not None:
        outs.append(("out", out))
    for i, (name, t) in enumerate(outs):
        for other, u in ins + outs[:i]:
            if _meet(_span(t), _span(u)):
                _require(other in ("x", "residual") and _same_rows(t, u),
                         f"{name} overlaps {other} and is not the same rows")


def spear_rms_norm(x, weight, eps: float = 1e-5, residual=None, residual_out=None, out=None,
                   out_format=None, stream=None):
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight over the last dimension of
    x [rows][hidden] (float16 or bfloat16) -> y, or (y, residual_out) with a residual; residual_out
    is h in x's type (give `residual` for it to update the residual in place).  y is of x's type, or
    a SpearMX where out_format is "fp4" or "fp8" or out is one."""
    import torch
    code, rows, hidden, x_stride = _matrix(x, "x", f32=False)
    device, shape = x.device, x.shape
    _as(weight, "weight", x.dtype, device, (hidden,))
    _require(residual is not None or residual_out is None, "residual_out without a residual")
    mx = isinstance(out, SpearMX) or (out is None and out_format is not None)
    r_stride = ro_stride = o_stride = 0
    if residual is not None:
        r_stride = _as(residual, "residual", x.dtype, device, shape)
    if residual_out is not None:
        ro_stride = _as(residual_out, "residual_out", x.dtype, device, shape)
    if out is not None:
        if mx:
            _require(out.device == device, f"out is on {out.device}, x on {device}")
            _require(out.shape == shape, f"out is {out.shape}, x {tuple(shape)}")
            _require(out_format is None or _format(out_format) == out.format, "out has another format")
        else:
            _require(out_format is None, "out_format with a 16-bit out")
            o_stride = _as(out, "out", x.dtype, device, shape)
    if out is not None or residual_out is not None:
        _norm_overlaps(x, weight, residual, residual_out, out, mx)
    _gpu(device)
    on = _On(device, stream)
    made = []
    if residual is not None and residual_out is None:
        residual_out = torch.empty(shape, dtype=x.dtype, device=device)
        ro_stride = hidden
        made.append(residual_out)
    if out is None:
        if mx:
            out = SpearMX.empty(rows, hidden, out_format, device)
            made.append(out._both)
        else:
            out = torch.empty(shape, dtype=x.dtype, device=device)
            o_stride = hidden
            made.append(out)
    if on.given and made:
        on.made(*made)
    args = SpearNormArgsC(code, rows, hidden, x.data_ptr(),
                          None if residual is None else residual.data_ptr(), weight.data_ptr(),
                          x_stride, r_stride, None if residual is None else residual_out.data_ptr(),
                          None if mx else out.data_ptr(), ro_stride, o_stride, out.at if mx else None, eps)
    with on as ptr:
        status = _lib().spear_rms_norm(ctypes.addressof(args), ptr)
    if status:
        _check(status)
    return out if residual is None else (out, residual_out)


def spear_mx_workspace_bytes(w: SpearMX, n_tokens: int) -> int:
    # (a count that does not fit the call's 32 bits as -1, which it takes as invalid)
    n_tokens = int(n_tokens)
    return int(_lib().spear_mx_workspace_bytes(w.at, n_tokens if 0 <= n_tokens < 2 ** 31 else -1))


def new_mx_workspace(w: SpearMX, n_tokens: int):
    """A 256-byte aligned workspace for products of w with at most n_tokens 16-bit tokens."""
    return _workspace(spear_mx_workspace_bytes(w, n_tokens), 0, w.device)


def _workspace(n: int, header: int, device):
    import torch
    if n == 0:
        raise SpearError(SPEAR_ERR_INVALID_ARGUMENT, "invalid sizes")
    buf = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    buf[off:off + header].zero_()
    return buf[off:off + n]


def _workspace_args(workspace, device):
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous() or workspace.device != device:
        raise ValueError(f"workspace must be contiguous and on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def spear_mx_linear(w: SpearMX, x, y=None, x_format="fp8", out_dtype=None, workspace=None, stream=None):
    """y [tokens][N] = x w^T for w [N][K] ("fp4") and x [tokens][K]: a SpearMX, or float16 or
    bfloat16 values, which are quantized to x_format in the workspace (these need one) first.  out_dtype: y's
    (None: x's, or bfloat16 for a SpearMX).  The header says how it is summed."""
    import torch
    device = w.device
    _require(x.device == device, f"x is on {x.device}, w on {device}")
    if isinstance(x, SpearMX):
        x_at, x_ptr, x_code, fmt, M, x_stride = x.at, None, 0, x.format, x.rows, 0
        K, dtype = x.cols, torch.bfloat16
    else:
        x_code, M, K, x_stride = _matrix(x, "x", f32=False)
        x_at, x_ptr, fmt, dtype = None, x.data_ptr(), _format(x_format), x.dtype
    if K != w.cols:
        raise ValueError(f"x has {K} columns, w {w.cols}")
    if y is not None:
        dtype = y.dtype if out_dtype is None else out_dtype
        y_stride = _as(y, "y", dtype, device, (M, w.rows))
        span = _span(y)
        _require(not _meets(w, span), "y must not overlap w")
        _require(not (_meets(x, span) if x_at else _meet(_span(x), span)), "y must not overlap x")
    elif out_dtype is not None:
        dtype = out_dtype
    code = _dtype_code(dtype, "out_dtype")
    ws, ws_bytes = _workspace_args(workspace, device)
    _gpu(device)
    on = _On(device, stream)
    if y is None:
        y = torch.empty((M, w.rows), dtype=dtype, device=device)
        y_stride = w.rows
        if on.given:
            on.made(y)
    if M == 0:
        return y
    args = SpearMXLinearArgsC(w.at, x_at, x_ptr, x_code, fmt, M, x_stride, y.data_ptr(), code, y_stride)
    with on as ptr:
        status = _lib().spear_mx_linear(ctypes.addressof(args), ws, ws_bytes, ptr)
    if status:
        _check(status)
    return y
