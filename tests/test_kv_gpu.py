"""The paged cache's operations (append, copy, fork, reserve, free, compact) against the oracle:
every result is bit-exact."""

import numpy as np
import pytest

from attn_helpers import DTYPES, as_layout, make_case, on_gpu
from gpu_helpers import note
from oracle import attn_ref
from quantized_gemm_error_amd import attn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy()


@pytest.mark.parametrize("layout", ["head", "token", "inside"])
@pytest.mark.parametrize("lens,chunks,heads,dim,page", [
    ([1], None, 1, 64, 16), ([5, 0, 16, 17, 300], None, 4, 128, 16), ([40], [40], 2, 128, 16),
    ([100, 7, 64, 33, 0], [50, 7, 0, 1, 0], 3, 64, 48), ([600, 256], [513, 3], 2, 128, 256),
])
def test_append(lens, chunks, heads, dim, page, layout):
    for dtype in DTYPES:
        note(f"append lens={lens} chunks={chunks} page={page} {layout} {dtype}")
        c = make_case(page, lens, (heads, heads), dim, page, dtype, chunks)
        c.table[0, 0] = c.table[0, 0] if len(lens) < 3 else -1  # a page out of range drops its tokens
        T = c.q.shape[0]
        gen = torch.Generator().manual_seed(7)
        fused = torch.randn((T, 2, heads, dim + 8), generator=gen).to(DTYPES[dtype]).cuda()
        k_new, v_new = fused[:, 0, :, :dim], fused[:, 1, :, 8:]
        k, v = as_layout(c.k, layout), as_layout(c.v, layout)
        attn.spear_kv_append(attn.SpearKVCache(k, v),
                             attn.SpearKVBatch(on_gpu(c.table), on_gpu(c.lens), on_gpu(c.starts)), k_new, v_new)
        torch.cuda.synchronize()
        for got, old, new in ((k, c.k, k_new), (v, c.v, v_new)):
            want = attn_ref.append_ref(bits(old).reshape(old.shape), bits(new).reshape(new.shape), c.table, lens, c.starts)
            assert np.array_equal(bits(got).reshape(old.shape), want)


def test_append_rows_before_position_zero_and_uncovered_rows():
    c = make_case(3, [8], (1, 1), 64, 16, "f16", [8])
    k, v = c.k.cuda(), c.v.cuda()
    new = torch.randn((10, 1, 64), dtype=torch.float16, device="cuda")  # rows 8 and 9 in no sequence
    attn.spear_kv_append(attn.SpearKVCache(k, v), attn.SpearKVBatch(on_gpu(c.table), on_gpu([5]), on_gpu([0, 8])), new, new)
    want = attn_ref.append_ref(bits(c.k).reshape(c.k.shape), bits(new).reshape(new.shape), c.table, [5], [0, 8])
    assert np.array_equal(bits(k).reshape(k.shape), want)


@pytest.mark.parametrize("layout", ["head", "token", "inside"])
@pytest.mark.parametrize("layers,heads,page,dim", [(1, 1, 16, 64), (3, 2, 16, 128), (2, 3, 48, 64), (40, 1, 32, 64)])
def test_copy_pages(layers, heads, page, dim, layout):
    gen = torch.Generator().manual_seed(page)
    P = 12
    host = torch.randn((2, layers, P, heads, page, dim), generator=gen).half()
    k, v = as_layout(host[0], layout), as_layout(host[1], layout)
    src, dst = [3, 3, 0, 11, -1, 5, 4, 12, 6], [1, 2, 10, 9, 8, 5, -2, 7, 99]
    attn.spear_kv_copy_pages(attn.SpearKVCache(k, v), on_gpu(src), on_gpu(dst))
    torch.cuda.synchronize()
    want = host.clone()
    for a, b in [(3, 1), (3, 2), (0, 10), (11, 9)]:
        want[:, :, b] = host[:, :, a]
    assert np.array_equal(bits(k), bits(want[0])) and np.array_equal(bits(v), bits(want[1]))


class Both:
    """A pool on the GPU and the oracle's, driven alike."""

    def __init__(self, pages, page_size, slots, width, layers=2, heads=2, dim=64, seed=0, layout="head"):
        gen = torch.Generator().manual_seed(seed)
        host = torch.randn((2, layers, pages, heads, page_size, dim), generator=gen).half()
        self.cache = attn.SpearKVCache(as_layout(host[0], layout), as_layout(host[1], layout))
        self.pool = attn.SpearKVPool.new(pages, page_size, slots, width)
        self.shape = host.shape
        per_page = bits(host).reshape(host.shape).transpose(2, 0, 1, 3, 4, 5)
        self.ref = attn_ref.PoolRef(np.zeros(pages, np.int32), np.full((slots, width), -1, np.int32),
                                    np.zeros(slots, np.int32), page_size, np.ascontiguousarray(per_page))

    def fork(self, src, dst):
        attn.spear_kv_fork(self.pool, on_gpu(src), on_gpu(dst))
        self.ref.fork(src, dst)

    def free(self, slots):
        attn.spear_kv_free(self.pool, on_gpu(slots))
        self.ref.free(slots)

    def reserve(self, slots, new_lens):
        missing = attn.spear_kv_reserve(self.pool, self.cache, on_gpu(slots), on_gpu(new_lens))
        want = self.ref.reserve(slots, new_lens)
        assert int(missing) == want
        return want

    def compact(self):
        used = attn.spear_kv_compact(self.pool, self.cache)
        assert int(used) == self.ref.compact()

    def check(self, what="", pages=True):
        torch.cuda.synchronize()
        assert np.array_equal(self.pool.refs.cpu().numpy(), self.ref.refs), f"{what}: refs"
        assert np.array_equal(self.pool.table.cpu().numpy(), self.ref.table), f"{what}: table"
        assert np.array_equal(self.pool.lens.cpu().numpy(), self.ref.lens), f"{what}: lens"
        if pages:
            want = self.ref.pages.transpose(1, 2, 0, 3, 4, 5)
            for i, t in enumerate((self.cache.k, self.cache.v)):
                assert np.array_equal(bits(t).reshape(want[i].shape), want[i]), f"{what}: pages"


@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("seed", range(4))
def test_random_pool_operations(seed, layout):
    rng = np.random.default_rng(seed)
    pages, S, slots, width = [(40, 16, 9, 7), (200, 32, 20, 9), (64, 48, 5, 300), (2500, 16, 30, 70)][seed]
    b = Both(pages, S, slots, width, seed=seed, layout=layout)
    for step in range(25):
        kind = rng.choice(["fork", "reserve", "reserve", "free", "compact"])
        note(f"pool seed={seed} step={step} {kind}")
        some = rng.permutation(slots)
        n = int(rng.integers(1, slots // 2 + 1))
        if kind == "fork":
            b.fork([int(rng.choice(some[n:])) for _ in range(n)], [int(s) for s in some[:n]])
        elif kind == "reserve":
            grow = [int(b.ref.lens[s]) + int(rng.integers(-3, min(width, 12) * S // 2)) for s in some[:n]]
            b.reserve([int(s) for s in some[:n]], [min(g, width * S) for g in grow])
        elif kind == "free":
            b.free([int(s) for s in some[:max(1, n // 2)]])
        else:
            b.compact()
        b.check(f"step {step} {kind}")


def test_many_children_of_one_page_and_the_last_holder_keeps_it():
    b = Both(300, 16, 101, 4)
    assert b.reserve([0], [21]) == 0
    b.fork([0] * 100, list(range(1, 101)))
    b.check("fork")
    assert b.reserve(list(range(101)), [22] * 101) == 0  # every holder writes: 100 copies
    b.check("reserve")
    assert int(b.pool.refs.max()) == 101                  # the full first page stays shared


def test_reserve_that_lacks_pages_or_names_nothing():
    b = Both(20, 16, 4, 30)
    assert b.reserve([0, 1], [100, 150]) == 0             # 7 + 10 pages
    assert b.reserve([2], [16 * 4]) == 1
    assert b.reserve([2, 3], [16 * 3, 16 * 5]) == 5
    assert b.reserve([2, 7], [1, 1]) == -1 and b.reserve([2, -1], [1, 1]) == -1
    assert b.reserve([2], [30 * 16 + 1]) == -1
    b.check("refused")
    assert b.reserve([2], [16 * 3]) == 0 and b.reserve([3], [1]) == 1
    assert b.reserve([], []) == 0 and b.reserve([0], [-4]) == 0
    b.check("full")


def test_fork_and_free_skip_slots_out_of_range():
    b = Both(30, 16, 4, 5)
    b.reserve([0, 1], [70, 20])
    b.fork([0, 9, -1, 1], [2, 3, 3, 1])
    b.free([4, -1, 1])
    b.check("skips")


@pytest.mark.parametrize("pages", [1, 1023, 1024, 1025, 5000])
def test_compact_pool_sizes(pages):
    """Small pages in large pools: nothing used, all used, every other page used, one far page."""
    b = Both(pages, 16, 3, 2500, layers=1, heads=1)
    b.compact()
    b.check("empty")
    if b.reserve([0], [16 * min(pages, 2500)]) == 0 and pages > 3:
        b.compact()
        keep = b.ref.table[0][: min(pages, 2500)].copy()
        for s, rows in ((1, keep[::2]), (2, keep[-1:])):
            row = np.full(2500, -1, np.int32)
            row[: len(rows)] = rows
            b.ref._row(s, row)
            b.ref.lens[s] = 16 * len(rows)
        for name in ("refs", "table", "lens"):
            getattr(b.pool, name).copy_(torch.from_numpy(getattr(b.ref, name)))
        b.free([0])
        b.compact()
        b.check("every other page")
        b.free([1])
        b.compact()
    b.check("far page")


@pytest.mark.parametrize("entries", [1, 2, 1000, 1024])
def test_reserve_entry_counts(entries):
    b = Both(4000, 16, 1024, 4, layers=1, heads=1)
    slots = list(np.random.default_rng(entries).permutation(1024)[:entries])
    assert b.reserve([int(s) for s in slots], [1 + (7 * int(s)) % 60 for s in slots]) == 0
    b.check("entries")


def test_graph_of_a_decode_step():
    """reserve, append and decode captured once and replayed for several steps, against the same
    calls made eagerly on a copy, with eager work between the replays."""
    H, D, S = 2, 64, 16

    def state():
        gen = torch.Generator(device="cuda").manual_seed(5)
        k, v = (torch.randn((40, H, S, D), generator=gen, device="cuda").half() for _ in range(2))
        pool = attn.SpearKVPool.new(40, S, 3, 8)
        cache = attn.SpearKVCache(k, v)
        attn.spear_kv_reserve(pool, cache, on_gpu([0, 1]), on_gpu([30, 14]))
        attn.spear_kv_fork(pool, on_gpu([1]), on_gpu([2]))
        return pool, cache

    x = torch.randn((3, 4 + 2 * H, D), device="cuda").half()
    slots, new_lens = on_gpu([0, 1, 2]), on_gpu([31, 15, 15])

    def step(pool, cache, ws):
        attn.spear_kv_reserve(pool, cache, slots, new_lens)
        batch = attn.SpearKVBatch(pool.table, pool.lens)
        attn.spear_kv_append(cache, batch, x[:, 4:4 + H], x[:, 4 + H:])
        return attn.spear_attn_decode(cache, batch, x[:, :4], workspace=ws)

    a, b = state(), state()
    ws = attn.new_attn_workspace(a[1], 4, 3, 3)
    spare = state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*spare, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*a, ws)
    for i in range(20):
        x.copy_(torch.randn_like(x))
        graph.replay()
        torch.cuda.synchronize()
        eager = step(*b, ws)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i
        for n in ("refs", "table", "lens"):
            assert torch.equal(getattr(a[0], n), getattr(b[0], n)), (i, n)
        new_lens += 1


@pytest.mark.parametrize("pages", [32768, 32769, 70000])
def test_compact_large_pools(pages):
    """Pools past the size up to which the counts are taken in one launch."""
    b = Both(pages, 16, 3, 4000, layers=1, heads=1)
    assert b.reserve([0, 1], [16 * 4000, 16 * 3000]) == 0
    far = np.random.default_rng(pages).choice(np.arange(7000, pages), 500, replace=False)
    row = np.full(4000, -1, np.int32)
    row[:500] = far
    b.ref._row(2, row)
    b.ref.lens[2] = 16 * 500
    for name in ("refs", "table", "lens"):
        getattr(b.pool, name).copy_(torch.from_numpy(getattr(b.ref, name)))
    b.free([0])
    b.compact()
    b.check("large pool")
