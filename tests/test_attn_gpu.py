"""Attention over the paged cache (spear_attn_decode, spear_attn_prefill) against the float64
oracle, elementwise, through the public binding."""

import math

import numpy as np
import pytest

from attn_helpers import Case, DTYPES, as_layout, check, make_case, on_gpu, reference
from gpu_helpers import note
from quantized_gemm_error_amd import attn, spear

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)


def run(c: Case, layout="head", window=0, sinks=0, scale=None, lse=True, call=None, ws=None, **kw):
    cache = attn.SpearKVCache(as_layout(c.k, layout), as_layout(c.v, layout))
    batch = attn.SpearKVBatch(on_gpu(c.table), on_gpu(c.lens), on_gpu(c.starts))
    q = kw.pop("q", None)
    q = c.q.cuda() if q is None else q
    if ws is None:
        ws = attn.new_attn_workspace(cache, q.shape[1], len(c.lens), q.shape[0])
    call = call or (attn.spear_attn_decode if c.starts is None else attn.spear_attn_prefill)
    return call(cache, batch, q, window=window, sinks=sinks, scale=scale, workspace=ws,
                return_lse=lse, **kw)


def verify(c, what, **kw):
    note(what)
    scale = kw.get("scale") or 1 / math.sqrt(c.q.shape[-1])
    out, lse = run(c, **kw)
    torch.cuda.synchronize()
    check(out, lse, reference(c, scale, kw.get("window", 0), kw.get("sinks", 0)), c, scale, what)


EDGE_LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [(1, 1), (4, 4), (8, 2), (7, 1), (24, 3), (16, 1), (20, 1), (33, 1)])
def test_decode_heads_and_lengths(heads, dim, dtype):
    c = make_case(heads[0] + dim, EDGE_LENS, heads, dim, 16, dtype)
    verify(c, f"decode heads={heads} dim={dim} {dtype}")


@pytest.mark.parametrize("layout", ["head", "token", "inside"])
@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 256])
def test_decode_pages_and_layouts(page, layout):
    c = make_case(page, [1, page - 1, page, page + 1, 3 * page + 5, 700, 0, 333], (8, 2), 128, page,
                  "bf16")
    verify(c, f"decode page={page} {layout}", layout=layout)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 16), (64, 0), (100, 37), (129, 32),
                                          (300, 500), (1000, 4), (0, 9)])
def test_decode_windows_and_sinks(window, sinks):
    c = make_case(window + sinks, [0, 1, 16, 33, 64, 100, 101, 137, 138, 257, 612, 999], (8, 2), 64, 16)
    verify(c, f"decode window={window} sinks={sinks}", window=window, sinks=sinks)


@pytest.mark.parametrize("lens,heads,dim", [
    ([6001], (8, 8), 128), ([4097, 5, 1200], (8, 1), 64), ([2049], (16, 2), 128), ([9000], (2, 2), 64),
    ([7] * 70 + [1500] + [31] * 70, (4, 2), 64),          # more sequences than lanes of a wave
    ([513 + 3 * i for i in range(40)], (4, 4), 128),
])
def test_decode_long_and_many(lens, heads, dim):
    c = make_case(sum(lens), lens, heads, dim, 16, "bf16")
    verify(c, f"decode lens={lens[:4]} heads={heads} dim={dim}")
    verify(c, f"decode lens={lens[:4]} heads={heads} dim={dim} window", window=700, sinks=5)


CHUNKS = [
    ([1], [1]), ([5], [5]), ([129], [129]), ([300], [1]), ([300], [37]), ([200, 64, 1, 77], [200, 1, 1, 13]),
    ([0, 40, 3], [0, 40, 2]), ([160, 128], [64, 128]), ([513], [130]), ([70] * 5, [1] * 5),
    ([9, 300], [0, 0]),
]


@pytest.mark.parametrize("lens,chunks", CHUNKS)
@pytest.mark.parametrize("heads,dim,dtype", [((4, 4), 128, "bf16"), ((8, 2), 64, "f16"), ((8, 1), 128, "f16"),
                                             ((6, 2), 64, "bf16"), ((5, 1), 128, "bf16")])
def test_chunk_shapes(lens, chunks, heads, dim, dtype):
    c = make_case(sum(lens) + dim, lens, heads, dim, 16, dtype, chunks)
    verify(c, f"chunk lens={lens} chunks={chunks} heads={heads} dim={dim} {dtype}")


@pytest.mark.parametrize("layout", ["head", "token", "inside"])
@pytest.mark.parametrize("page", [16, 48, 64, 256])
def test_chunk_pages_and_layouts(page, layout):
    c = make_case(page + 1, [page + 1, 3 * page + 5, 301], (4, 2), 128, page, "bf16", [page, 70, 150])
    verify(c, f"chunk page={page} {layout}", layout=layout)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (64, 0), (65, 70), (100, 37), (300, 2), (0, 5)])
def test_chunk_windows_and_sinks(window, sinks):
    c = make_case(window + sinks, [700, 130, 90], (4, 1), 64, 16, "f16", [140, 130, 1])
    verify(c, f"chunk window={window} sinks={sinks}", window=window, sinks=sinks)
    c = make_case(window + sinks, [400], (2, 2), 128, 32, "bf16", [300])
    verify(c, f"chunk dim=128 window={window} sinks={sinks}", window=window, sinks=sinks)


@pytest.mark.parametrize("lens,chunks,heads", [([3001], [40], (4, 1)), ([2500, 700], [9, 3], (2, 2))])
def test_chunk_few_rows_over_a_long_cache(lens, chunks, heads):
    c = make_case(lens[0], lens, heads, 128, 16, "bf16", chunks)
    verify(c, f"chunk lens={lens} chunks={chunks}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_one_row_chunks_equal_decode(dtype):
    lens = [0, 1, 33, 200, 611]
    c = make_case(3, lens, (8, 2), 128, 16, dtype)
    verify(c, "chunk call without q_starts", call=attn.spear_attn_prefill)


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("chunks", [None, [20, 33, 1, 0]])
def test_slots_without_tokens_do_not_matter(fill, chunks):
    lens = [20, 33, 100, 0]
    for dim in (64, 128):
        c = make_case(9, lens, (8, 2), dim, 16, "bf16", chunks, unused=fill)
        verify(c, f"unused slots hold {fill}, chunks={chunks} dim={dim}")


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2)])
def test_hidden_positions_do_not_matter(fill, dim, heads):
    """Later rows of the chunk and what the window leaves out hold no numbers; the rows that see
    none of those give what they give without them."""
    for window, sinks, bad in [(0, 0, [150, 155, 180]), (40, 3, [5, 60, 61, 70])]:
        c = make_case(11, [200], heads, dim, 16, "bf16", [100])
        scale = 1 / math.sqrt(dim)
        clean = reference(c, scale, window, sinks)
        for j in bad:
            for t in (c.k, c.v):
                t[c.table[0, j // 16], :, j % 16] = fill
        note(f"hidden positions hold {fill}: window={window} dim={dim} heads={heads}")
        out, lse = run(c, window=window, sinks=sinks)
        torch.cuda.synchronize()
        sees = [r for r in range(100)
                if any((j <= 100 + r) and (not window or 100 + r - j < window or j < sinks) for j in bad)]
        rows = [r for r in range(100) if r not in sees]
        assert len(rows) >= 50 and len(sees) >= 10
        part = Case(c.q[rows], c.k, c.v, c.table, c.lens, None, c.dtype)
        check(out[rows], lse[rows], [a[rows] for a in clean], part, scale, "rows that see only numbers")
        if math.isnan(fill):  # and a row that does see one has no number
            assert torch.isnan(out[sees]).any(-1).all()


def test_decode_window_hides_what_is_not_a_number():
    c = make_case(4, [300, 90], (8, 2), 128, 16, "f16")
    ref = reference(c, 1 / math.sqrt(128), 40, 3)
    for b, j in [(0, 5), (0, 200), (0, 259), (1, 3), (1, 49)]:
        for t in (c.k, c.v):
            t[c.table[b, j // 16], :, j % 16] = float("nan")
    out, lse = run(c, window=40, sinks=3)
    check(out, lse, ref, c, 1 / math.sqrt(128), "decode, hidden NaN")


@pytest.mark.parametrize("chunks", [None, [30, 90]])
def test_pages_out_of_range_hide_their_tokens(chunks):
    for window, sinks in ((0, 0), (100, 20)):
        c = make_case(6, [300, 90], (8, 2), 128, 16, "f16", chunks)
        c.table[0, 2], c.table[0, 7], c.table[1, 0], c.table[1, 5] = -1, 1 << 30, -7, len(c.k)
        verify(c, f"bad pages chunks={chunks} window={window}", window=window, sinks=sinks)
    c.table[:] = -1
    out, lse = run(c)
    assert not out.any() and torch.isneginf(lse).all()


def test_lengths_out_of_range_are_bounded():
    c = make_case(6, [64, 64], (4, 2), 64, 16, "f16")
    c.table = np.ascontiguousarray(c.table[:, :4])
    c.lens = [10 ** 6, -5]
    out, lse = run(c)
    c.lens = [64, 0]
    check(out, lse, reference(c, 1 / 8, 0, 0), c, 1 / 8, "bounded lengths")


def test_rows_past_the_cached_length_see_nothing():
    c = make_case(8, [5], (4, 2), 64, 16, "bf16", [5])
    c.lens = [3]  # rows 0 and 1 lie before position 0
    verify(c, "rows before position 0")


@pytest.mark.parametrize("chunks", [None, [40, 1, 20]])
@pytest.mark.parametrize("dim", [64, 128])
def test_strided_queries_and_outputs(chunks, dim):
    c = make_case(2, [40, 300, 71], (8, 2), dim, 16, "f16", chunks)
    T = c.q.shape[0]
    scale = 1 / math.sqrt(dim)
    ref = reference(c, scale, 0, 0)
    fused = torch.full((T, 8 * dim + 24), float("nan"), dtype=c.q.dtype, device="cuda")
    q = fused[:, 16:16 + 8 * dim].unflatten(1, (8, dim))
    q.copy_(c.q)
    for out in (torch.empty((8, T, dim), dtype=q.dtype, device="cuda").transpose(0, 1),
                torch.full((T, 9, dim + 8), 7.0, dtype=q.dtype, device="cuda")[:, 1:, :dim]):
        got, lse = run(c, q=q, out=out)
        assert got is out
        check(got, lse, ref, c, scale, "strided")
    one = c.q[:, :1].cuda().expand(T, 8, dim)  # the same query for every head
    c.q = one.cpu().contiguous()
    got, lse = run(c, q=one)
    check(got, lse, reference(c, scale, 0, 0), c, scale, "broadcast query")


@pytest.mark.parametrize("chunks", [None, [3, 30]])
def test_scales_and_large_scores(chunks):
    c = make_case(12, [70, 333], (4, 2), 128, 16, "f16", chunks)
    verify(c, "scale 0.01", scale=0.01)
    verify(c, "negative scale", scale=-0.3)
    c = make_case(12, [70, 333], (4, 2), 128, 16, "f16", chunks, gain=40)
    verify(c, "scores in the hundreds", scale=0.25)


@pytest.mark.parametrize("chunks", [None, [50, 1, 120]])
def test_a_workspace_serves_many_calls_with_equal_results(chunks):
    """The same call gives the same bits, also after calls of other sizes in the same workspace."""
    c = make_case(31, [2000, 900, 150], (8, 2), 64, 16, "bf16", chunks)
    other = make_case(32, [10, 3000], (8, 2), 64, 16, "bf16", None if chunks is None else [10, 77])
    cache = attn.SpearKVCache(c.k.cuda(), c.v.cuda())
    ws = attn.new_attn_workspace(cache, 8, 3, 171)
    first = run(c, ws=ws)
    for i in range(10):
        run(other, ws=ws, window=(0, 500)[i % 2])
        again = run(c, ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(first, again)), i
    verify(c, "workspace reuse", ws=ws)
    verify(other, "workspace reuse, other sizes", ws=ws)


@pytest.mark.parametrize("chunks", [None, [50, 1, 120]])
def test_on_another_stream(chunks):
    c = make_case(33, [800, 900, 150], (8, 2), 128, 16, "bf16", chunks)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = run(c, stream=side)
    side.synchronize()
    check(out, lse, reference(c, 1 / math.sqrt(128), 0, 0), c, 1 / math.sqrt(128), "side stream")


@pytest.mark.parametrize("chunks", [None, [50, 1, 120]])
def test_graph_replays(chunks):
    """A captured call follows the values its buffers hold at each replay; eager calls and
    synchronizations lie between the replays."""
    cases = [make_case(40 + i, lens, (8, 2), 64, 16, "f16", chunks, spare=s)
             for i, (lens, s) in enumerate([([1500, 64, 120], 3), ([1490, 63, 121], 3), ([1489, 50, 123], 3)])]
    assert len({c.k.shape for c in cases}) == 1 and len({c.table.shape for c in cases}) == 1
    c = cases[0]
    k, v, q, table, lens = c.k.cuda(), c.v.cuda(), c.q.cuda(), on_gpu(c.table), on_gpu(c.lens)
    cache, batch = attn.SpearKVCache(k, v), attn.SpearKVBatch(table, lens, on_gpu(c.starts))
    ws = attn.new_attn_workspace(cache, 8, 3, q.shape[0])
    call = attn.spear_attn_decode if chunks is None else attn.spear_attn_prefill
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(cache, batch, q, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = call(cache, batch, q, workspace=ws, return_lse=True)
    for i in range(7):
        c = cases[i % 3]
        for t, x in ((k, c.k), (v, c.v), (q, c.q), (table, on_gpu(c.table)), (lens, on_gpu(c.lens))):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        check(out, lse, reference(c, 1 / 8, 0, 0), c, 1 / 8, f"replay {i}")
        eager = call(cache, batch, q, workspace=ws)
        assert torch.equal(eager, out), i


def test_offsets_past_32_bits():
    """Pages far apart in one array: their offsets in elements and bytes pass 2^32."""
    c = make_case(50, [100, 40], (8, 2), 128, 16, "f16", spare=0)
    P = c.k.shape[0]
    step = (1 << 32) // (P - 1) // 8 * 8 + 8
    big = torch.empty(step * (P - 1) + 2 * 2 * 16 * 128, dtype=torch.float16, device="cuda")
    views = [torch.as_strided(big, c.k.shape, (step, 16 * 128, 128, 1), o * 2 * 16 * 128) for o in (0, 1)]
    for t, x in zip(views, (c.k, c.v)):
        t.copy_(x)
    cache = attn.SpearKVCache(*views)
    for chunks in (None, [60, 7]):
        q = c.q if chunks is None else torch.randn((67, 8, 128), generator=torch.Generator().manual_seed(1)).half()
        cc = Case(q, c.k, c.v, c.table, c.lens, None if chunks is None else [0, 60, 67], "f16")
        batch = attn.SpearKVBatch(on_gpu(cc.table), on_gpu(cc.lens), on_gpu(cc.starts))
        ws = attn.new_attn_workspace(cache, 8, 2, q.shape[0])
        call = attn.spear_attn_decode if chunks is None else attn.spear_attn_prefill
        out, lse = call(cache, batch, q.cuda(), workspace=ws, return_lse=True)
        check(out, lse, reference(cc, 1 / math.sqrt(128), 0, 0), cc, 1 / math.sqrt(128), "far pages")


@pytest.mark.parametrize("heads", [(2, 2), (8, 1)])
def test_many_short_sequences(heads):
    """More sequences than a few waves' lanes, of none, one and a few new tokens."""
    rng = np.random.default_rng(heads[0])
    lens = [int(n) for n in rng.integers(0, 70, 600)]
    lens[77], lens[400] = 2000, 1300
    c = make_case(5, lens, heads, 64, 16, "f16")
    verify(c, "decode, 600 sequences")
    c = make_case(6, lens, heads, 64, 16, "bf16", [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 4, 600))])
    verify(c, "chunks, 600 sequences")
    verify(c, "chunks, 600 sequences, window", window=20, sinks=3)


def test_rows_of_no_sequence_are_left_alone():
    c = make_case(7, [40, 60], (4, 2), 64, 16, "f16", [10, 20])
    q = torch.cat([c.q, c.q[:5]]).cuda()  # five rows past q_starts' end
    out = torch.full_like(q, 9.0)
    run(c, q=q, out=out, lse=False)
    check(out[:30], None, reference(c, 1 / 8, 0, 0), c, 1 / 8, "covered rows")
    assert (out[30:] == 9).all()


@pytest.mark.parametrize("starts", [[0, 50, 20], [7, 3, 1 << 30], [-5, 10, 99], [0, 0, -1], [1 << 30, 5, 30]])
def test_q_starts_out_of_order_stay_inside(starts):
    """Nothing outside the tensors is touched: what lies beside q and out keeps its values."""
    c = make_case(7, [40, 60], (4, 2), 64, 16, "f16", [10, 20])
    c.starts = starts
    frame = torch.full((90, 4, 64), 5.0, dtype=torch.float16, device="cuda")
    out = frame[30:60]
    run(c, out=out, lse=False)
    torch.cuda.synchronize()
    assert (frame[:30] == 5).all() and (frame[60:] == 5).all()


def test_no_rows_and_no_sequences():
    c = make_case(1, [5, 9], (4, 2), 64, 16, "f16", [0, 0])
    out, lse = run(c)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    cache = attn.SpearKVCache(c.k.cuda(), c.v.cuda())
    batch = attn.SpearKVBatch(torch.empty((0, 3), dtype=torch.int32, device="cuda"),
                              torch.empty(0, dtype=torch.int32, device="cuda"))
    assert attn.spear_attn_decode(cache, batch, torch.empty((0, 4, 64), dtype=torch.float16, device="cuda")
                                  ).shape == (0, 4, 64)


def test_refusals_on_the_gpu():
    c = make_case(1, [50, 9], (4, 2), 64, 16, "f16")
    with pytest.raises(spear.SpearError, match="multiple of n_kv_heads"):
        run(c, q=torch.zeros((2, 3, 64), dtype=torch.float16, device="cuda"), ws=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"))
    with pytest.raises(spear.SpearError, match="window"):
        run(c, window=-1)
    with pytest.raises(spear.SpearError, match="scale"):
        run(c, scale=float("inf"))


# Chunks of whole blocks of rows that do not fill the chip: the tiles of a block are shared out
# inside a workgroup and, with more of them, among workgroups; odd and even numbers of tiles.
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 5), (1100, 0)])
@pytest.mark.parametrize("lens,chunks", [([577], [140]), ([2111], [200]), ([1800, 640, 1300], [257, 128, 99]),
                                         ([4001], [128]), ([1500, 900], [130, 900])])
@pytest.mark.parametrize("heads,dim,dtype", [((2, 2), 128, "bf16"), ((4, 1), 64, "f16")])
def test_chunks_of_few_blocks_over_long_caches(heads, dim, dtype, lens, chunks, window, sinks):
    c = make_case(sum(lens), lens, heads, dim, 16, dtype, chunks)
    verify(c, f"chunk lens={lens} chunks={chunks} window={window} {dtype}", window=window, sinks=sinks)


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("length", [700, 1237, 1300, 2113])
@pytest.mark.parametrize("dim", [64, 128])
def test_hidden_positions_of_few_blocks_over_long_caches(fill, length, dim):
    """What only the window's first tiles and the chunk's last ones hold, as above."""
    n = 150
    past = length - n
    for window, bad in [(0, [length - 1, length - 20, past + 100]), (513, [past - 512, past - 470, length - 2])]:
        c = make_case(length, [length], (2, 2), dim, 16, "bf16", [n])
        scale = 1 / math.sqrt(dim)
        clean = reference(c, scale, window, 0)
        for j in bad:
            for t in (c.k, c.v):
                t[c.table[0, j // 16], :, j % 16] = fill
        note(f"hidden positions hold {fill}: length={length} window={window} dim={dim}")
        out, lse = run(c, window=window)
        torch.cuda.synchronize()
        sees = [r for r in range(n)
                if any(j <= past + r and (not window or past + r - j < window) for j in bad)]
        rows = [r for r in range(n) if r not in sees]
        assert len(rows) >= 50 and len(sees) >= 10
        part = Case(c.q[rows], c.k, c.v, c.table, c.lens, None, c.dtype)
        check(out[rows], lse[rows], [a[rows] for a in clean], part, scale, "rows that see only numbers")
        if math.isnan(fill):
            assert torch.isnan(out[sees]).any(-1).all()
