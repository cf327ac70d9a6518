"""Binding of libspear's paged key-value cache and attention (include/spear_attn.h), same names
as the C ABI.

Argument marshalling and checks only, as in spear.py: every step runs in the library's HIP
kernels, and there is no fallback.  The handles (SpearKVCache, SpearKVBatch, SpearKVPool) check
their tensors once and keep the C structs; a program makes the cache's and the pool's once and the
batch's once per step, for all layers.  They hold references to their tensors and read no values
from them.
"""

from __future__ import annotations

import ctypes
import math

from . import spear
from .spear import SpearError, _check, _require, SPEAR_ERR_INVALID_ARGUMENT

SPEAR_ATTN_MAX_SEQS = 4096
SPEAR_KV_MAX_ENTRIES = 1024
SPEAR_ATTN_HEADER_BYTES = 16384

# Every function the header declares, for the export check.
EXPORTED = (
    "spear_attn_workspace_bytes", "spear_attn_decode", "spear_attn_prefill", "spear_kv_append",
    "spear_kv_copy_pages", "spear_kv_scratch_words", "spear_kv_fork", "spear_kv_reserve",
    "spear_kv_free", "spear_kv_compact",
)

_P, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class SpearKVCacheC(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("dtype", _i32), ("n_layers", _i32), ("num_pages", _i32),
                ("n_kv_heads", _i32), ("page_size", _i32), ("head_dim", _i32),
                ("stride_layer", _i64), ("stride_page", _i64), ("stride_head", _i64),
                ("stride_token", _i64)]


class SpearKVBatchC(ctypes.Structure):
    _fields_ = [("n_seqs", _i32), ("table_width", _i32), ("n_tokens", _i32),
                ("block_table", _P), ("kv_lens", _P), ("q_starts", _P)]


class SpearAttnArgsC(ctypes.Structure):
    _fields_ = [("n_q_heads", _i32), ("window", _i32), ("sinks", _i32), ("scale", ctypes.c_float),
                ("q", _P), ("q_stride_token", _i64), ("q_stride_head", _i64),
                ("out", _P), ("out_stride_token", _i64), ("out_stride_head", _i64), ("lse", _P)]


class SpearKVPoolC(ctypes.Structure):
    _fields_ = [("num_pages", _i32), ("page_size", _i32), ("n_slots", _i32), ("table_width", _i32),
                ("refs", _P), ("table", _P), ("lens", _P), ("scratch", _P)]


_bound = None


def load_library():
    """libspear.so with this header's functions declared (raises if it has not been built)."""
    global _bound
    if _bound is not None:
        return _bound
    lib = spear.load_library()
    C, B, A = (ctypes.POINTER(t) for t in (SpearKVCacheC, SpearKVBatchC, SpearAttnArgsC))
    L = ctypes.POINTER(SpearKVPoolC)
    lib.spear_attn_workspace_bytes.argtypes = [C, _i32, _i32, _i32]
    lib.spear_attn_workspace_bytes.restype = _sz
    lib.spear_attn_decode.argtypes = [C, B, A, _P, _sz, _P]
    lib.spear_attn_prefill.argtypes = [C, B, A, _P, _sz, _P]
    lib.spear_kv_append.argtypes = [C, B, _P, _P, _i64, _i64, _i64, _i64, _P]
    lib.spear_kv_copy_pages.argtypes = [C, _P, _P, _i32, _P]
    lib.spear_kv_scratch_words.argtypes = [_i32, _i32, _i32]
    lib.spear_kv_scratch_words.restype = _sz
    lib.spear_kv_fork.argtypes = [L, _P, _P, _i32, _P]
    lib.spear_kv_reserve.argtypes = [L, C, _P, _P, _i32, _P, _P]
    lib.spear_kv_free.argtypes = [L, _P, _i32, _P]
    lib.spear_kv_compact.argtypes = [L, C, _P, _P]
    for name in EXPORTED:
        if name not in ("spear_attn_workspace_bytes", "spear_kv_scratch_words"):
            getattr(lib, name).restype = _i32
    _bound = lib
    return lib


def _lib():
    return _bound if _bound is not None else load_library()


def _int32(t, name: str, dim: int, device=None) -> None:
    import torch
    if (t is not None and t.dtype is torch.int32 and t.dim() == dim and t.is_contiguous()
            and (device is None or t.device == device)):
        return
    _require(t is not None, f"{name} is missing")
    _require(t.dtype == torch.int32, f"{name} has dtype {t.dtype}, expected torch.int32", TypeError)
    _require(t.dim() == dim and t.is_contiguous(), f"{name} must be a contiguous {dim}-D tensor")
    raise ValueError(f"{name} is on {t.device}, expected {device}")


_INT32_MIN, _INT32_MAX = -2 ** 31, 2 ** 31 - 1


def _fits(value: int, name: str) -> int:
    """value, which ctypes would cut to its low 32 bits if it did not fit them."""
    if not _INT32_MIN <= value <= _INT32_MAX:
        raise ValueError(f"{name}={value} does not fit in 32 bits")
    return value


def _gpu(device) -> None:
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")


class _On:
    """The stream a call runs on; its device is made the current one for the call."""

    def __init__(self, device, stream):
        import torch
        self.given = stream is not None
        if stream is None:
            # (the handle alone where torch offers it: a Stream object costs 2 us)
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            self.ptr = raw(device.index) if raw else torch.cuda.current_stream(device).cuda_stream
        else:
            self.stream = stream
            self.ptr = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
        self.guard = None if torch.cuda.current_device() == device.index else \
            torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.ptr

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def made(self, *tensors):
        """Tensors allocated by the call (on the current stream) and written on the given one."""
        import torch
        st, device = self.stream, tensors[0].device
        if not hasattr(st, "cuda_stream"):  # a raw handle: of the tensors' device
            st = torch.cuda.ExternalStream(st, device=device) if st else torch.cuda.default_stream(device)
        here = torch.cuda.current_stream(device)
        if st.cuda_stream != here.cuda_stream:
            st.wait_stream(here)  # what the memory served before ends first
            for t in tensors:
                t.record_stream(st)


class SpearKVCache:
    """The pages of one layer ([pages][kv heads][page][dim]) or of all layers (a leading layer
    dimension): k and v, float16 or bfloat16, of the same shape and strides, the last dimension
    contiguous.  Token-major pages are the transposed view of a [pages][page][heads][dim] tensor."""

    def __init__(self, k, v):
        code = spear._dtype_code(k)
        _require(k.dim() in (4, 5), f"k must be [pages][heads][page][dim] or have a leading layer "
                                    f"dimension, got {k.dim()}-D")
        _require(k.shape == v.shape and k.stride() == v.stride() and k.dtype == v.dtype,
                 "k and v must agree in shape, strides and dtype")
        _require(k.device == v.device, f"k is on {k.device}, v on {v.device}")
        _require(k.numel() > 0, "the cache is empty")
        _require(k.stride(-1) == 1, "the last dimension of the cache must be contiguous")
        shape, strides = tuple(k.shape), k.stride()
        if k.dim() == 4:
            shape, strides = (1,) + shape, (0,) + strides
        _require(max(shape) < 2 ** 31, f"cache of shape {tuple(k.shape)} is too large")
        self.k, self.v, self.device = k, v, k.device
        self.n_layers, self.num_pages, self.n_kv_heads, self.page_size, self.head_dim = shape
        self.dtype, self.scale = k.dtype, 1.0 / math.sqrt(self.head_dim)
        self.spans = _span(k), _span(v)
        self.c = SpearKVCacheC(k.data_ptr(), v.data_ptr(), code, *shape, *strides[:4])
        self.ref = ctypes.byref(self.c)

    def layer(self, i: int) -> "SpearKVCache":
        """The cache of layer i, for the attention and append calls."""
        _require(self.k.dim() == 5, "the cache has no layer dimension")
        return SpearKVCache(self.k[i], self.v[i])


class SpearKVBatch:
    """The sequences of one step (int32 device tensors): block_table [seqs][width], kv_lens [seqs]
    with the step's tokens included, q_starts [seqs + 1] or None for one token each."""

    def __init__(self, block_table, kv_lens, q_starts=None):
        _int32(block_table, "block_table", 2)
        self.device = block_table.device
        _int32(kv_lens, "kv_lens", 1, self.device)
        n, width = block_table.shape
        _require(kv_lens.numel() == n, f"kv_lens has {kv_lens.numel()} entries, block_table {n} rows")
        _require(width >= 1, "block_table has no columns")
        if q_starts is not None:
            _int32(q_starts, "q_starts", 1, self.device)
            _require(q_starts.numel() == n + 1, f"q_starts has {q_starts.numel()} entries, expected {n + 1}")
        self.block_table, self.kv_lens, self.q_starts = block_table, kv_lens, q_starts
        self.n_seqs = n
        self.ref = ctypes.byref(SpearKVBatchC(n, width, n, block_table.data_ptr(), kv_lens.data_ptr(),
                                              None if q_starts is None else q_starts.data_ptr()))

    @property
    def c(self) -> SpearKVBatchC:
        return self.ref._obj

    def rows(self, n_tokens: int):
        """The C struct for a call with this many rows (kept: a step's calls have as many).
        Structs are never written once others can see them, so threads may share a batch."""
        ref = self.ref
        if n_tokens != ref._obj.n_tokens:
            c = SpearKVBatchC.from_buffer_copy(ref._obj)
            c.n_tokens = _fits(n_tokens, "rows")
            self.ref = ref = ctypes.byref(c)
        return ref


class SpearKVPool:
    """The pages' bookkeeping (int32 device tensors): refs [pages], table [slots][width], lens
    [slots]; see spear_kv_pool_t.  Allocates its scratch."""

    def __init__(self, refs, table, lens, page_size: int):
        import torch
        _int32(refs, "refs", 1)
        self.device = refs.device
        _int32(table, "table", 2, self.device)
        _int32(lens, "lens", 1, self.device)
        _require(lens.numel() == table.shape[0], f"lens has {lens.numel()} entries, table {table.shape[0]} rows")
        _require(refs.numel() > 0 and table.numel() > 0, "the pool is empty")
        n_slots, width = table.shape
        page_size = _fits(int(page_size), "page_size")
        words = int(load_library().spear_kv_scratch_words(refs.numel(), n_slots, width))
        if words == 0:
            raise SpearError(SPEAR_ERR_INVALID_ARGUMENT, "invalid pool sizes")
        self.refs, self.table, self.lens, self.page_size = refs, table, lens, page_size
        self.scratch = torch.empty(words, dtype=torch.int32, device=self.device)
        self.c = SpearKVPoolC(refs.numel(), self.page_size, n_slots, width, refs.data_ptr(),
                              table.data_ptr(), lens.data_ptr(), self.scratch.data_ptr())
        self.ref = ctypes.byref(self.c)

    @classmethod
    def new(cls, num_pages: int, page_size: int, n_slots: int, table_width: int, device="cuda"):
        """A pool whose pages are all free."""
        import torch
        return cls(torch.zeros(num_pages, dtype=torch.int32, device=device),
                   torch.full((n_slots, table_width), -1, dtype=torch.int32, device=device),
                   torch.zeros(n_slots, dtype=torch.int32, device=device), page_size)


def spear_attn_workspace_bytes(cache: SpearKVCache, n_q_heads: int, n_seqs: int, n_tokens: int) -> int:
    # (sizes that do not fit the call's 32 bits as the nearest that do, which it takes as invalid)
    sizes = (max(-1, min(int(n), _INT32_MAX)) for n in (n_q_heads, n_seqs, n_tokens))
    return int(load_library().spear_attn_workspace_bytes(cache.ref, *sizes))


def new_attn_workspace(cache: SpearKVCache, n_q_heads: int, n_seqs: int, n_tokens: int):
    """A 256-byte aligned workspace with a zeroed header for attention calls of at most these sizes."""
    import torch
    n = spear_attn_workspace_bytes(cache, n_q_heads, n_seqs, n_tokens)
    if n == 0:
        raise SpearError(SPEAR_ERR_INVALID_ARGUMENT, spear.spear_last_error())
    buf = torch.empty(n + 256, dtype=torch.uint8, device=cache.device)
    off = (-buf.data_ptr()) % 256
    buf[off:off + SPEAR_ATTN_HEADER_BYTES].zero_()
    return buf[off:off + n]


def _rows(t, name: str, cache, tokens=None, heads=None):
    """t is [tokens][heads][head_dim] of the cache's dtype, its last dimension contiguous -> its
    sizes and strides.  (One test for all on the call path; the message is found afterwards.)"""
    if t.dim() == 3:
        (T, H, D), (st, sh, sd) = t.shape, t.stride()
        if (D == cache.head_dim and sd == 1 and t.dtype is cache.dtype and t.device == cache.device
                and (tokens is None or T == tokens) and (heads is None or H == heads)):
            return T, H, st, sh
    _require(t.dim() == 3, f"{name} must be [tokens][heads][head_dim], got {t.dim()}-D")
    _require(t.dtype == cache.dtype, f"{name} has dtype {t.dtype}, the cache {cache.dtype}", TypeError)
    _require(t.shape[2] == cache.head_dim and (tokens is None or t.shape[0] == tokens)
             and (heads is None or t.shape[1] == heads),
             f"{name} has shape {tuple(t.shape)}, expected "
             f"({'any' if tokens is None else tokens}, {'any' if heads is None else heads}, {cache.head_dim})")
    _require(t.stride(2) == 1, f"the last dimension of {name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, the cache on {cache.device}")


def _span(t):
    """The addresses of a tensor's first byte and past its last one."""
    at = t.data_ptr()
    if t.numel() == 0:
        return at, at
    return at, at + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))


def _meet(a, b) -> bool:
    return a[0] < b[1] and b[0] < a[1]


def _attention(fn, cache, batch, q, out, scale, window, sinks, workspace, return_lse, stream, decode):
    import torch
    T, Hq, q_tok, q_head = _rows(q, "q", cache)
    device = cache.device
    if batch.device != device:
        raise ValueError(f"the batch is on {batch.device}, the cache on {device}")
    if batch.q_starts is None:
        if T != batch.n_seqs:
            raise ValueError(f"q has {T} rows for {batch.n_seqs} sequences of one token")
    elif decode:
        raise ValueError("decode takes one token per sequence: the batch has q_starts")
    if out is not None:
        _, _, o_tok, o_head = _rows(out, "out", cache, T, Hq)
        span = _span(out)
        _require(not _meet(span, _span(q)), "out must not overlap q")
        _require(not _meet(span, cache.spans[0]) and not _meet(span, cache.spans[1]),
                 "out must not overlap the cache")
    ws, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_contiguous() or workspace.device != device:
            raise ValueError(f"workspace must be contiguous and on {device}")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _fits(window, "window"), _fits(sinks, "sinks")
    _gpu(device)
    on = _On(device, stream)
    made = []
    if out is None:
        out = torch.empty((T, Hq, cache.head_dim), dtype=cache.dtype, device=device)
        o_tok, o_head = Hq * cache.head_dim, cache.head_dim
        made.append(out)
    lse = None
    if return_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=device)
        made.append(lse)
    if on.given and made:
        on.made(*made)
    args = SpearAttnArgsC(Hq, window, sinks, cache.scale if scale is None else scale,
                          q.data_ptr(), q_tok, q_head, out.data_ptr(), o_tok, o_head,
                          None if lse is None else lse.data_ptr())
    with on as ptr:
        status = fn(cache.ref, batch.rows(T), ctypes.byref(args), ws, ws_bytes, ptr)
    if status:
        _check(status)
    return (out, lse) if return_lse else out


def spear_attn_decode(cache: SpearKVCache, batch: SpearKVBatch, q, out=None, scale=None,
                      window: int = 0, sinks: int = 0, workspace=None, return_lse: bool = False,
                      stream=None):
    """q [seqs][heads][dim] -> out of the same shape (and lse [seqs][heads] when asked for).
    scale None: 1 / sqrt(dim).  window 0: none."""
    return _attention(_lib().spear_attn_decode, cache, batch, q, out, scale, window, sinks,
                      workspace, return_lse, stream, True)


def spear_attn_prefill(cache: SpearKVCache, batch: SpearKVBatch, q, out=None, scale=None,
                       window: int = 0, sinks: int = 0, workspace=None, return_lse: bool = False,
                       stream=None):
    """q [tokens][heads][dim], rows as in the batch's q_starts -> out of the same shape."""
    return _attention(_lib().spear_attn_prefill, cache, batch, q, out, scale, window, sinks,
                      workspace, return_lse, stream, False)


def spear_kv_append(cache: SpearKVCache, batch: SpearKVBatch, k, v, stream=None) -> None:
    """Store new keys and values [tokens][kv heads][dim] in the batch's pages."""
    T, _, k_tok, k_head = _rows(k, "k", cache, heads=cache.n_kv_heads)
    _, _, v_tok, v_head = _rows(v, "v", cache, T, cache.n_kv_heads)
    if batch.device != cache.device:
        raise ValueError(f"the batch is on {batch.device}, the cache on {cache.device}")
    if batch.q_starts is None and T != batch.n_seqs:
        raise ValueError(f"k has {T} rows for {batch.n_seqs} sequences of one token")
    for span in (_span(k), _span(v)):
        if _meet(span, cache.spans[0]) or _meet(span, cache.spans[1]):
            raise ValueError("k and v must not overlap the cache")
    _gpu(cache.device)
    with _On(cache.device, stream) as ptr:
        status = _lib().spear_kv_append(cache.ref, batch.rows(T), k.data_ptr(), v.data_ptr(), k_tok, k_head,
                                        v_tok, v_head, ptr)
    if status:
        _check(status)


def spear_kv_copy_pages(cache: SpearKVCache, src, dst, stream=None) -> None:
    """Page src[i] to page dst[i] of all layers (int32 device tensors)."""
    _int32(src, "src", 1, cache.device)
    _int32(dst, "dst", 1, cache.device)
    if src.numel() != dst.numel():
        raise ValueError(f"src has {src.numel()} entries, dst {dst.numel()}")
    _gpu(cache.device)
    with _On(cache.device, stream) as ptr:
        _check(_lib().spear_kv_copy_pages(cache.ref, src.data_ptr(), dst.data_ptr(),
                                                  src.numel(), ptr))


def spear_kv_fork(pool: SpearKVPool, src, dst, stream=None) -> None:
    """Slots dst[i] become copies of slots src[i] that share their pages."""
    _int32(src, "src", 1, pool.device)
    _int32(dst, "dst", 1, pool.device)
    if src.numel() != dst.numel():
        raise ValueError(f"src has {src.numel()} entries, dst {dst.numel()}")
    _gpu(pool.device)
    with _On(pool.device, stream) as ptr:
        _check(_lib().spear_kv_fork(pool.ref, src.data_ptr(), dst.data_ptr(), src.numel(), ptr))


def spear_kv_reserve(pool: SpearKVPool, cache: SpearKVCache, slots, new_lens, missing=None,
                     stream=None):
    """Pages for slots to hold new_lens tokens, copy on write -> missing, an int32 device tensor
    [1]: 0, or how many pages lack (then nothing was changed), or -1 for an invalid entry."""
    import torch
    _int32(slots, "slots", 1, pool.device)
    _int32(new_lens, "new_lens", 1, pool.device)
    if slots.numel() != new_lens.numel():
        raise ValueError(f"slots has {slots.numel()} entries, new_lens {new_lens.numel()}")
    if cache.device != pool.device:
        raise ValueError(f"the cache is on {cache.device}, the pool on {pool.device}")
    if missing is not None:
        _int32(missing, "missing", 1, pool.device)
        _require(missing.numel() == 1, "missing must hold one value")
    _gpu(pool.device)
    on = _On(pool.device, stream)
    if missing is None:
        missing = torch.empty(1, dtype=torch.int32, device=pool.device)
        if on.given:
            on.made(missing)
    with on as ptr:
        _check(_lib().spear_kv_reserve(pool.ref, cache.ref, slots.data_ptr(),
                                               new_lens.data_ptr(), slots.numel(),
                                               missing.data_ptr(), ptr))
    return missing


def spear_kv_free(pool: SpearKVPool, slots, stream=None) -> None:
    """Release the pages of slots."""
    _int32(slots, "slots", 1, pool.device)
    _gpu(pool.device)
    with _On(pool.device, stream) as ptr:
        _check(_lib().spear_kv_free(pool.ref, slots.data_ptr(), slots.numel(), ptr))


def spear_kv_compact(pool: SpearKVPool, cache: SpearKVCache, used=None, stream=None):
    """Move the used pages to the lowest indices -> used, an int32 device tensor [1]: how many."""
    import torch
    if cache.device != pool.device:
        raise ValueError(f"the cache is on {cache.device}, the pool on {pool.device}")
    if used is not None:
        _int32(used, "used", 1, pool.device)
        _require(used.numel() == 1, "used must hold one value")
    _gpu(pool.device)
    on = _On(pool.device, stream)
    if used is None:
        used = torch.empty(1, dtype=torch.int32, device=pool.device)
        if on.given:
            on.made(used)
    with on as ptr:
        _check(_lib().spear_kv_compact(pool.ref, cache.ref, used.data_ptr(), ptr))
    return used
