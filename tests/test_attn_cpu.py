"""The attention and cache entry points without a GPU: the exports, the C ABI's refusals (before
any launch), workspace and scratch sizes, and the binding's checks on CPU tensors."""

import ctypes
import os
import re

import pytest

from quantized_gemm_error_amd import attn, spear

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(spear.LIB_PATH):
        pytest.fail("libspear.so is not built: run python -m quantized_gemm_error_amd.build")
    return attn.load_library()


def test_exports_every_declared_function(lib):
    text = open(os.path.join(ROOT, "include", "spear_attn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = set(re.findall(r"\b(spear_(?:attn|kv)_[a-z0-9_]+)\s*\(", text))
    assert declared == set(attn.EXPORTED)
    for name in declared:
        assert hasattr(lib, name), name


def _cache(**kw):
    f = dict(k=1 << 32, v=1 << 33, dtype=0, n_layers=1, num_pages=10, n_kv_heads=2, page_size=16, head_dim=64,
             stride_layer=0, stride_page=2 * 16 * 64, stride_head=16 * 64, stride_token=64)
    f.update(kw)
    return attn.SpearKVCacheC(*[f[n] for n, _ in attn.SpearKVCacheC._fields_])


def _batch(**kw):
    f = dict(n_seqs=3, table_width=4, n_tokens=3, block_table=1 << 34, kv_lens=1 << 35, q_starts=None)
    f.update(kw)
    return attn.SpearKVBatchC(*[f[n] for n, _ in attn.SpearKVBatchC._fields_])


def _args(**kw):
    f = dict(n_q_heads=8, window=0, sinks=0, scale=0.1, q=1 << 36, q_stride_token=512, q_stride_head=64,
             out=1 << 37, out_stride_token=512, out_stride_head=64, lse=None)
    f.update(kw)
    return attn.SpearAttnArgsC(*[f[n] for n, _ in attn.SpearAttnArgsC._fields_])


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
R = ctypes.byref

BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=(1 << 32) + 8), INVALID), (dict(dtype=2), INVALID),
    (dict(n_layers=0), INVALID), (dict(num_pages=0), INVALID), (dict(n_kv_heads=0), INVALID),
    (dict(page_size=0), INVALID), (dict(page_size=24), UNSUPPORTED), (dict(page_size=1 << 17), UNSUPPORTED),
    (dict(head_dim=80), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(n_kv_heads=2000, stride_page=1 << 30), UNSUPPORTED),
    (dict(stride_token=60), INVALID), (dict(stride_page=0), INVALID), (dict(stride_head=64), INVALID),
    (dict(stride_page=2 * 16 * 64 - 8), INVALID), (dict(stride_token=-64), INVALID),
    (dict(stride_page=1 << 62), INVALID),
    (dict(stride_token=1 << 26, stride_page=1 << 32, stride_head=64), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_refusals(lib, kw, status):
    c = _cache(**kw)
    for fn in (lib.spear_attn_decode, lib.spear_attn_prefill):
        assert fn(R(c), R(_batch()), R(_args()), None, 0, None) == status
    assert lib.spear_kv_append(R(c), R(_batch()), 1 << 36, 1 << 37, 128, 64, 128, 64, None) == status
    assert lib.spear_kv_copy_pages(R(c), 1 << 36, 1 << 37, 1, None) == status
    assert lib.spear_attn_workspace_bytes(R(c), 8, 3, 3) == 0
    assert spear.spear_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(n_seqs=-1), INVALID), (dict(table_width=0), INVALID), (dict(n_tokens=-1), INVALID),
    (dict(n_tokens=4), INVALID), (dict(block_table=None), INVALID), (dict(kv_lens=None), INVALID),
    (dict(kv_lens=(1 << 35) + 2), INVALID), (dict(n_seqs=5000, n_tokens=5000), UNSUPPORTED),
    (dict(table_width=1 << 27), UNSUPPORTED), (dict(n_seqs=4096, n_tokens=4096, table_width=1 << 20), UNSUPPORTED),
])
def test_batch_refusals(lib, kw, status):
    b = _batch(**kw)
    for fn in (lib.spear_attn_decode, lib.spear_attn_prefill):
        assert fn(R(_cache()), R(b), R(_args()), None, 0, None) == status
    assert lib.spear_kv_append(R(_cache()), R(b), 1 << 36, 1 << 37, 128, 64, 128, 64, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n_q_heads=0), INVALID), (dict(n_q_heads=7), INVALID), (dict(n_q_heads=8192), UNSUPPORTED),
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q=(1 << 36) + 4), INVALID),
    (dict(q_stride_token=-512), INVALID), (dict(q_stride_head=60), INVALID), (dict(out_stride_token=0), INVALID),
    (dict(out_stride_head=32), INVALID), (dict(out_stride_token=8 * 64 - 8), INVALID), (dict(out=1 << 36), INVALID),
    (dict(lse=(1 << 38) + 1), INVALID),
])
def test_argument_refusals(lib, kw, status):
    for fn in (lib.spear_attn_decode, lib.spear_attn_prefill):
        assert fn(R(_cache()), R(_batch()), R(_args(**kw)), None, 0, None) == status


def test_too_many_rows(lib):
    b = _batch(n_tokens=1 << 24, q_starts=1 << 39)
    c = _cache(n_kv_heads=1, stride_head=0)
    assert lib.spear_attn_prefill(R(c), R(b), R(_args(n_q_heads=128)), None, 0, None) == UNSUPPORTED
    b = _batch(n_tokens=(1 << 24) + 1, q_starts=1 << 39)
    assert lib.spear_kv_append(R(c), R(b), 1 << 36, 1 << 37, 128, 64, 128, 64, None) == UNSUPPORTED


def test_null_structs_layers_and_q_starts(lib):
    assert lib.spear_attn_decode(None, R(_batch()), R(_args()), None, 0, None) == INVALID
    assert lib.spear_attn_decode(R(_cache()), None, R(_args()), None, 0, None) == INVALID
    assert lib.spear_attn_decode(R(_cache()), R(_batch()), None, None, 0, None) == INVALID
    assert lib.spear_attn_decode(R(_cache()), R(_batch(q_starts=1 << 38)), R(_args()), None, 0, None) == INVALID
    two = _cache(n_layers=2, stride_layer=10 * 2 * 16 * 64)
    assert lib.spear_attn_prefill(R(two), R(_batch()), R(_args()), None, 0, None) == INVALID
    assert lib.spear_kv_append(R(two), R(_batch()), 1 << 36, 1 << 37, 128, 64, 128, 64, None) == INVALID


def test_calls_without_rows_launch_nothing(lib):
    empty = _batch(n_seqs=0, n_tokens=0, block_table=None, kv_lens=None)
    for fn in (lib.spear_attn_decode, lib.spear_attn_prefill):
        assert fn(R(_cache()), R(empty), R(_args(q=None, out=None)), None, 0, None) == 0
    assert lib.spear_kv_append(R(_cache()), R(empty), None, None, 0, 0, 0, 0, None) == 0
    assert lib.spear_kv_copy_pages(R(_cache()), None, None, 0, None) == 0


def test_append_refusals(lib):
    for a in [(None, 1 << 37, 128, 64, 128, 64), (1 << 36, None, 128, 64, 128, 64), (8, 1 << 37, 128, 64, 128, 64),
              (1 << 36, 1 << 37, 100, 64, 128, 64), (1 << 36, 1 << 37, 128, 64, 128, -64)]:
        assert lib.spear_kv_append(R(_cache()), R(_batch()), *a, None) == INVALID


def test_workspace_sizes_grow_and_are_asked_for(lib):
    sizes = [lib.spear_attn_workspace_bytes(R(_cache()), 8, n, n) for n in (0, 1, 8, 64, 512, 4096)]
    assert all(s > 0 for s in sizes) and sizes == sorted(sizes)
    for bad in [(7, 3, 3), (0, 3, 3), (8, -1, 3), (8, 3, -1), (8, 5000, 3)]:
        assert lib.spear_attn_workspace_bytes(R(_cache()), *bad) == 0


def _pool(**kw):
    f = dict(num_pages=10, page_size=16, n_slots=4, table_width=5, refs=1 << 32, table=1 << 33, lens=1 << 34, scratch=1 << 35)
    f.update(kw)
    return attn.SpearKVPoolC(*[f[n] for n, _ in attn.SpearKVPoolC._fields_])


@pytest.mark.parametrize("kw,status", [
    (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(n_slots=0), INVALID), (dict(table_width=0), INVALID),
    (dict(refs=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(scratch=None), INVALID),
    (dict(table=(1 << 33) + 1), INVALID), (dict(num_pages=1 << 25), UNSUPPORTED), (dict(n_slots=1 << 20, table_width=1 << 12), UNSUPPORTED),
])
def test_pool_refusals(lib, kw, status):
    p, a, b = _pool(**kw), 1 << 36, 1 << 37
    assert lib.spear_kv_fork(R(p), a, b, 1, None) == status
    assert lib.spear_kv_free(R(p), a, 1, None) == status
    assert lib.spear_kv_reserve(R(p), R(_cache()), a, b, 1, 1 << 38, None) == status
    assert lib.spear_kv_compact(R(p), R(_cache()), 1 << 38, None) == status


def test_list_refusals(lib):
    p, c, a, b = _pool(), _cache(), 1 << 36, 1 << 37
    assert lib.spear_kv_fork(R(p), None, b, 1, None) == INVALID
    assert lib.spear_kv_fork(R(p), a, b, -1, None) == INVALID
    assert lib.spear_kv_fork(R(p), None, None, 0, None) == 0
    assert lib.spear_kv_free(R(p), a + 2, 1, None) == INVALID
    assert lib.spear_kv_free(R(p), None, 0, None) == 0
    assert lib.spear_kv_reserve(R(p), R(c), a, b, 1025, 1 << 38, None) == INVALID
    assert lib.spear_kv_reserve(R(p), R(c), a, b, 1, None, None) == INVALID
    assert lib.spear_kv_reserve(R(p), R(_cache(num_pages=11)), a, b, 1, 1 << 38, None) == INVALID
    assert lib.spear_kv_compact(R(p), R(_cache(page_size=32, stride_page=2 * 32 * 64, stride_head=32 * 64)), 1 << 38, None) == INVALID
    assert lib.spear_kv_compact(R(p), R(c), None, None) == INVALID
    assert lib.spear_kv_copy_pages(R(c), a, b, -1, None) == INVALID
    assert lib.spear_kv_copy_pages(R(c), a, None, 1, None) == INVALID


def test_scratch_words(lib):
    assert lib.spear_kv_scratch_words(0, 1, 1) == 0 and lib.spear_kv_scratch_words(10, 0, 1) == 0
    small, large = (lib.spear_kv_scratch_words(n, 4, 5) for n in (10, 100000))
    assert 3 * 10 < small and 3 * 100000 + 98 < large


# ------------------------------------------------------------------ the binding, on CPU tensors

def _t(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype)


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _handles():
    return attn.SpearKVCache(_t(10, 2, 16, 64), _t(10, 2, 16, 64)), attn.SpearKVBatch(_i(3, 4), _i(3))


def test_valid_cpu_tensors_fail_only_on_the_device(lib):
    cache, batch = _handles()
    pool = attn.SpearKVPool(_i(10), _i(3, 4), _i(3), 16)
    for call in [lambda: attn.spear_attn_decode(cache, batch, _t(3, 8, 64)),
                 lambda: attn.spear_attn_prefill(cache, attn.SpearKVBatch(_i(3, 4), _i(3), _i(4)), _t(9, 8, 64)),
                 lambda: attn.spear_kv_append(cache, batch, _t(3, 2, 64), _t(3, 2, 64)),
                 lambda: attn.spear_kv_copy_pages(cache, _i(2), _i(2)),
                 lambda: attn.spear_kv_fork(pool, _i(2), _i(2)), lambda: attn.spear_kv_free(pool, _i(2)),
                 lambda: attn.spear_kv_reserve(pool, cache, _i(2), _i(2)),
                 lambda: attn.spear_kv_compact(pool, cache)]:
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.parametrize("k,v,exc", [
    (_t(10, 2, 64), _t(10, 2, 64), ValueError), (_t(10, 2, 16, 64), _t(10, 2, 16, 32), ValueError),
    (_t(10, 2, 16, 64), _t(10, 16, 2, 64).transpose(1, 2), ValueError),
    (_t(10, 2, 16, 64), _t(10, 2, 16, 64, dtype=torch.bfloat16), ValueError),
    (_t(10, 2, 16, 64, dtype=torch.float32), _t(10, 2, 16, 64, dtype=torch.float32), TypeError),
    (_t(10, 2, 64, 16).transpose(2, 3), _t(10, 2, 64, 16).transpose(2, 3), ValueError),
    (_t(0, 2, 16, 64), _t(0, 2, 16, 64), ValueError),
])
def test_bad_caches(k, v, exc):
    with pytest.raises(exc):
        attn.SpearKVCache(k, v)


@pytest.mark.parametrize("args,exc", [
    ((_i(3), _i(3)), ValueError), ((_i(3, 4), _i(4)), ValueError), ((_i(3, 4), _i(3), _i(3)), ValueError),
    ((_i(4, 3).t(), _i(3)), ValueError), ((_i(3, 4).long(), _i(3)), TypeError), ((_i(3, 4), _i(3).long()), TypeError),
    ((_i(3, 0), _i(3)), ValueError), ((None, _i(3)), ValueError),
])
def test_bad_batches(args, exc):
    with pytest.raises(exc):
        attn.SpearKVBatch(*args)


@pytest.mark.parametrize("q,out,exc", [
    (_t(2, 8, 64), None, ValueError), (_t(3, 8, 128), None, ValueError), (_t(3, 512), None, ValueError),
    (_t(3, 8, 64, dtype=torch.bfloat16), None, TypeError), (_t(3, 64, 8).transpose(1, 2), None, ValueError),
    (_t(3, 8, 64), _t(3, 7, 64), ValueError), (_t(3, 8, 64), _t(3, 8, 64, dtype=torch.float32), TypeError),
])
def test_bad_queries_and_outputs(q, out, exc):
    cache, batch = _handles()
    with pytest.raises(exc):
        attn.spear_attn_decode(cache, batch, q, out=out)


def test_out_may_not_overlap_its_inputs():
    cache, batch = _handles()
    q = _t(3, 8, 64)
    with pytest.raises(ValueError, match="overlap q"):
        attn.spear_attn_decode(cache, batch, q, out=q)
    with pytest.raises(ValueError, match="overlap the cache"):
        attn.spear_attn_decode(cache, batch, q, out=cache.k.flatten()[:3 * 512].view(3, 8, 64))
    with pytest.raises(ValueError, match="overlap the cache"):
        attn.spear_kv_append(cache, batch, cache.v.flatten()[:384].view(3, 2, 64), _t(3, 2, 64))


def test_decode_refuses_chunks_and_pools_their_shapes(lib):
    cache, _ = _handles()
    with pytest.raises(ValueError, match="q_starts"):
        attn.spear_attn_decode(cache, attn.SpearKVBatch(_i(3, 4), _i(3), _i(4)), _t(3, 8, 64))
    for bad in [(_i(10), _i(3, 4), _i(4)), (_i(10), _i(12), _i(3)), (_i(0), _i(3, 4), _i(3))]:
        with pytest.raises(ValueError):
            attn.SpearKVPool(*bad, 16)
    pool = attn.SpearKVPool(_i(10), _i(3, 4), _i(3), 16)
    with pytest.raises(ValueError):
        attn.spear_kv_fork(pool, _i(2), _i(3))
    with pytest.raises(ValueError):
        attn.spear_kv_reserve(pool, cache, _i(2), _i(3))
    with pytest.raises(ValueError):
        attn.spear_kv_compact(pool, cache, used=_i(2))
    with pytest.raises(TypeError):
        attn.spear_kv_free(pool, _i(2).long())


def test_layers_of_a_cache():
    k, v = _t(3, 10, 2, 16, 64), _t(3, 10, 2, 16, 64)
    cache = attn.SpearKVCache(k, v)
    assert cache.n_layers == 3 and cache.layer(1).k.data_ptr() == k[1].data_ptr()
    with pytest.raises(ValueError):
        cache.layer(1).layer(0)


class _Stream:
    def __init__(self, handle, log):
        self.cuda_stream, self.log = handle, log

    def wait_stream(self, other):
        self.log.append(("wait", self.cuda_stream, other.cuda_stream))


@pytest.mark.parametrize("given", [0, 77, "object"])
def test_memory_made_for_a_given_stream_waits_on_the_tensors_device(monkeypatch, given):
    """A raw handle is taken as a stream of the tensors' device, not of the current one."""
    log, asked = [], []

    def named(name, handle):
        def make(*args, device=None):
            asked.append((name, args, device))
            return _Stream(args[0] if name == "external" else handle, log)
        return make

    device = torch.device("cuda", 1)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=None: named("external", 0)(ptr, device=device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: named("default", 0)(device=device))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: named("current", 5)(device=device))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)

    class Made:
        def record_stream(self, stream):
            log.append(("record", stream.cuda_stream))

    made = Made()
    made.device = device
    stream = _Stream(9, log) if given == "object" else given
    handle = 9 if given == "object" else given
    attn._On(device, stream).made(made)
    assert log == [("wait", handle, 5), ("record", handle)]
    assert asked and all(d == device for _, _, d in asked), asked


@pytest.mark.parametrize("after", ["c", "ref"])
def test_threads_that_share_a_batch_get_their_own_row_counts(after):
    """Another thread's call with another number of rows, between the steps of this one's."""
    import threading

    class Interrupted(attn.SpearKVBatch):
        between = None

        def __setattr__(self, name, value):
            super().__setattr__(name, value)
            if name == after and self.between is not None:
                call, self.between = self.between, None
                other = threading.Thread(target=call)
                other.start()
                other.join()

    batch, theirs = Interrupted(_i(3, 4), _i(3), _i(4)), []
    batch.between = lambda: theirs.append(batch.rows(50))
    mine = batch.rows(20)
    assert mine._obj.n_tokens == 20 and all(r._obj.n_tokens == 50 for r in theirs)
    for n in (50, 20, 50, 7):
        assert batch.rows(n)._obj.n_tokens == n and batch.rows(n)._obj.n_seqs == 3


@pytest.mark.parametrize("kw", [dict(window=2 ** 32 + 100), dict(window=2 ** 31), dict(sinks=2 ** 32), dict(sinks=2 ** 63),
                                dict(window=-(2 ** 32) + 7), dict(sinks=-(2 ** 31) - 1)])
def test_windows_and_sinks_past_the_types_range(lib, kw):
    """Refused, not cut to their low 32 bits."""
    cache, batch = _handles()
    chunk = attn.SpearKVBatch(_i(3, 4), _i(3), _i(4))
    for call, b in ((attn.spear_attn_decode, batch), (attn.spear_attn_prefill, chunk)):
        with pytest.raises(ValueError, match=next(iter(kw))):
            call(cache, b, _t(3, 8, 64), **kw)


def test_page_sizes_and_counts_past_the_types_range(lib):
    for size in (2 ** 32 + 16, 2 ** 31):
        with pytest.raises(ValueError, match="page_size"):
            attn.SpearKVPool(_i(10), _i(3, 4), _i(3), size)
    cache, _ = _handles()
    assert attn.spear_attn_workspace_bytes(cache, 8, 3, 3) > 0
    for bad in ((2 ** 32 + 8, 3, 3), (8, 2 ** 32 + 3, 3), (8, 3, 2 ** 32 + 3)):
        assert attn.spear_attn_workspace_bytes(cache, *bad) == 0
    many = _t(1, 2, 64).expand(2 ** 32 + 3, 2, 64)
    with pytest.raises(ValueError):
        attn.spear_kv_append(cache, attn.SpearKVBatch(_i(3, 4), _i(3), _i(4)), many, many)
    with pytest.raises(ValueError, match="rows"):
        attn.SpearKVBatch(_i(3, 4), _i(3), _i(4)).rows(2 ** 32 + 3)


def test_more_entries_than_slots_are_refused(lib):
    """They cannot be distinct, and their pages could be more than the plan's 32-bit sums hold."""
    p, c, a, b = _pool(n_slots=4), _cache(), 1 << 36, 1 << 37
    assert lib.spear_kv_reserve(R(p), R(c), a, b, 5, 1 << 38, None) == INVALID
    assert "5" in spear.spear_last_error()
