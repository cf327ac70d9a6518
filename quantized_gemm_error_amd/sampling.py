"""Binding of libspear's sampling (include/spear_sample.h), same names as the C ABI.

Argument marshalling and checks only, as in spear.py: the draw runs in the library's HIP kernels,
and there is no fallback.
"""

from __future__ import annotations

import ctypes

from . import spear
from .attn import _gpu, _meet, _On, _span
from .mx import _dtype_code, _matrix, _workspace, _workspace_args
from .spear import _check, _require

SPEAR_SAMPLE_HEADER_BYTES = 16384

# Every function the header declares, for the export check.
EXPORTED = ("spear_sample_workspace_bytes", "spear_sample")

_P, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class SpearSampleArgsC(ctypes.Structure):
    _fields_ = [("logits", _P), ("dtype", _i32), ("rows", _i32), ("vocab", _i32), ("stride", _i64),
                ("u", _P), ("temperature", _P), ("top_k", _P), ("top_p", _P), ("min_p", _P),
                ("tokens", _P), ("logprobs", _P)]


_bound = None


def load_library():
    """libspear.so with this header's functions declared (raises if it has not been built)."""
    global _bound
    if _bound is not None:
        return _bound
    lib = spear.load_library()
    lib.spear_sample_workspace_bytes.argtypes = [_i32, _i32]
    lib.spear_sample_workspace_bytes.restype = _sz
    lib.spear_sample.argtypes = [_P, _P, _sz, _P]
    lib.spear_sample.restype = _i32
    _bound = lib
    return lib


def _lib():
    return _bound if _bound is not None else load_library()


def spear_sample_workspace_bytes(rows: int, vocab: int) -> int:
    # (sizes that do not fit the call's 32 bits as -1, which it takes as invalid)
    rows, vocab = (int(n) if 0 <= int(n) < 2 ** 31 else -1 for n in (rows, vocab))
    return int(_lib().spear_sample_workspace_bytes(rows, vocab))


def new_sample_workspace(rows: int, vocab: int, device="cuda"):
    """A 256-byte aligned workspace with a zeroed header for calls of at most these sizes."""
    return _workspace(spear_sample_workspace_bytes(rows, vocab), SPEAR_SAMPLE_HEADER_BYTES, device)


def _per_row(t, name: str, rows: int, dtype, device):
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != (rows,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of {rows} values, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t.data_ptr()


def spear_sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None,
                 workspace=None, return_logprobs: bool = False, stream=None):
    """A token of each row of logits [rows][vocab] (float16, bfloat16 or float32) from the random
    numbers u [rows] in [0, 1) -> tokens [rows] (int32), and the logarithms of their shares of what
    is kept when asked for.  temperature, top_p, min_p: float32 [rows]; top_k: int32 [rows]; None:
    1, no limit.  The header says which tokens are kept and in which order."""
    import torch
    code, rows, vocab, stride = _matrix(logits, "logits")
    device, f32 = logits.device, torch.float32
    _require(u is not None, "u is missing")
    at = [_per_row(u, "u", rows, f32, device), _per_row(temperature, "temperature", rows, f32, device),
          _per_row(top_k, "top_k", rows, torch.int32, device), _per_row(top_p, "top_p", rows, f32, device),
          _per_row(min_p, "min_p", rows, f32, device)]
    if tokens is not None:
        _per_row(tokens, "tokens", rows, torch.int32, device)
        for t, name in ((logits, "logits"), (u, "u"), (temperature, "temperature"), (top_k, "top_k"),
                        (top_p, "top_p"), (min_p, "min_p")):
            _require(t is None or not _meet(_span(tokens), _span(t)), f"tokens must not overlap {name}")
    ws, ws_bytes = _workspace_args(workspace, device)
    _gpu(device)
    on = _On(device, stream)
    made = []
    if tokens is None:
        tokens = torch.empty(rows, dtype=torch.int32, device=device)
        made.append(tokens)
    logprobs = None
    if return_logprobs:
        logprobs = torch.empty(rows, dtype=f32, device=device)
        made.append(logprobs)
    if on.given and made:
        on.made(*made)
    if rows:
        args = SpearSampleArgsC(logits.data_ptr(), code, rows, vocab, stride, *at, tokens.data_ptr(),
                                None if logprobs is None else logprobs.data_ptr())
        with on as ptr:
            status = _lib().spear_sample(ctypes.addressof(args), ws, ws_bytes, ptr)
        if status:
            _check(status)
    return (tokens, logprobs) if return_logprobs else tokens
