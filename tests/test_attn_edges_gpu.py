"""Attention and cache calls at the ends of their arguments' ranges (window, scale, size of the
scores, values that are not finite, q_starts past the rows), against the float64 oracle."""

import math

import numpy as np
import pytest

from attn_helpers import Case, DTYPES, check, f64, make_case, on_gpu, reference
from gpu_helpers import note
from oracle import attn_ref
from quantized_gemm_error_amd import attn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)


def run(c: Case, window=0, sinks=0, scale=None):
    cache = attn.SpearKVCache(c.k.cuda(), c.v.cuda())
    batch = attn.SpearKVBatch(on_gpu(c.table), on_gpu(c.lens), on_gpu(c.starts))
    ws = attn.new_attn_workspace(cache, c.q.shape[1], len(c.lens), c.q.shape[0])
    call = attn.spear_attn_decode if c.starts is None else attn.spear_attn_prefill
    out, lse = call(cache, batch, c.q.cuda(), window=window, sinks=sinks, scale=scale, workspace=ws,
                    return_lse=True)
    torch.cuda.synchronize()
    return out, lse


# Shapes that take the forms of the kernels: one token a sequence; a chunk of one group of waves; of
# two groups; of blocks cut into parts whose sums meet in memory; single rows cut into parts.
SHAPES = [([5, 40, 1500, 3001], None), ([200, 70], [100, 1]), ([1300], [150]), ([4001], [128]), ([2900, 33], [1, 1])]


# ---------------------------------------------------------------------------------- windows

@pytest.mark.parametrize("lens,chunks,heads", [([5], [8], (4, 2)), ([0, 5, 700], [3, 9, 140], (4, 2)),
                                               ([600, 5], [200, 12], (2, 2)), ([2000], [130], (2, 2)),
                                               ([0, 1, 33, 700], None, (4, 2))])
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 6, 3), (7, 2 ** 31 - 1)])
def test_windows_and_sinks_at_the_types_limit(lens, chunks, heads, window, sinks):
    """As large as the type holds, rows before position 0 among them."""
    note(f"window={window} sinks={sinks} lens={lens} chunks={chunks}")
    c = make_case(3, lens, heads, 64, 16, "f16", chunks)
    out, lse = run(c, window, sinks)
    check(out, lse, reference(c, 1 / 8, window, sinks), c, 1 / 8, "window at the limit")


# --------------------------------------------------------------------- the softmax's tail

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,chunks", [([500], None), ([4097], None), ([700], [100]), ([4097], [3]), ([32768], [1]),
                                         ([32768], [130])])
@pytest.mark.parametrize("depth", [8.0, 12.0, 16.0, 17.5, 19.0])
def test_many_keys_far_below_one_with_the_value_zero(depth, lens, chunks, dtype):
    """The first key has the weight 1 and the value 0, every other one e^-depth and 1: the result
    is their number times that weight, not what is left of it in the type's subnormal numbers.

    A weight is rounded to the type relative to its own size (h), or where it falls below fp16's
    normal range by at most 2^-25, 2^-38 against the row's largest."""
    note(f"tail depth={depth} lens={lens} chunks={chunks} {dtype}")
    c = make_case(1, lens, (2, 1), 64, 16, dtype, chunks)
    n = 1 if chunks is None else chunks[0]
    c.q.zero_(), c.k.zero_(), c.v.fill_(1)
    c.q[..., 0] = depth
    c.k[c.table[0, 0], :, 0, 0] = 1
    c.v[c.table[0, 0], :, 0] = 0
    out, lse = run(c, scale=1.0)
    h = torch.finfo(DTYPES[dtype]).eps / 2
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    seen = lens[0] - n + 1 + np.arange(n)[:, None]
    w = math.exp(-depth)
    want = np.broadcast_to((seen - 1) * w / (1 + (seen - 1) * w), (n, 2))
    # scores are exact, their exponent's factor log2 e and the exponential are good to 2^-20
    rel = 2 * h + 2.0 ** -19 + seen * 2.0 ** -24
    tol = rel * want + tiny * (2.0 ** -13 * (seen - 1) / (1 + (seen - 1) * w) + 1)
    err = np.abs(f64(out) - want[..., None])
    assert (err <= tol[..., None]).all(), (float(f64(out)[-1, 0, 0]), float(want[-1, 0]))
    z = depth + np.log1p((seen - 1) * w)
    assert (np.abs(f64(lse) - z) <= 2.0 ** -18 + 2.0 ** -21 * z).all()


# ---------------------------------------------------------------------- the size of scores

def equal_scores(dtype, shape, a, b, heads=(4, 2)):
    """A case of shape `shape` whose keys score a b exactly or, two of three, 3/4 |a b| less."""
    lens, chunks = shape
    c = make_case(7, lens, heads, 64, 16, dtype, chunks)
    c.q.zero_(), c.k.zero_()
    c.q[..., 0] = a
    top = torch.arange(c.k.shape[2]) % 3 == 0
    c.k[..., 0] = torch.where(top, b, b - abs(0.75 * b)).to(c.k.dtype)
    return c


def check_equal_scores(c, scale, a, b):
    """Where differences of scores are hundreds or more a row is the mean of the values of the keys
    with the largest one, whose scores are one exact product: weights are 1 or 0, each rounding of
    them is one of h, of the result another; the sums add 2^-20 and count 2^-24."""
    out, lse = run(c, scale=scale)
    a, b = (float(torch.tensor(x, dtype=c.k.dtype)) for x in (a, b))
    h = torch.finfo(c.k.dtype).eps / 2
    S, G, got, z, values = c.k.shape[2], c.q.shape[1] // c.k.shape[1], f64(out), f64(lse), f64(c.v)
    starts = list(range(len(c.lens) + 1)) if c.starts is None else c.starts
    for s, length in enumerate(c.lens):
        n = starts[s + 1] - starts[s]
        for i in range(n):
            j = np.arange(length - n + i + 1)
            j = j[(j % S) % 3 == 0]
            v = values[c.table[s, j // S], :, j % S]
            for head in range(c.q.shape[1]):
                vv = v[:, head // G]
                tol = (2 * h + 2.0 ** -20 + len(j) * 2.0 ** -24) * np.abs(vv).mean(0) + 2.0 ** -25
                err = np.abs(got[starts[s] + i, head] - vv.mean(0))
                assert (err <= tol).all(), (s, i, head, err.max())
                want = scale * a * b + math.log(len(j))
                assert abs(z[starts[s] + i, head] - want) <= 2.0 ** -21 * abs(want)


@pytest.mark.parametrize("dtype,scale,a,b", [
    ("f16", 0.125, 6e4, 6e4), ("f16", 1.0, 2e4, 2.4e4), ("f16", 1.0, 3e4, 5e4), ("f16", 1.0, 4.5e4, -3.3e4), ("f16", 1e4, 700, 900),
    ("bf16", 1.0, 6e4, 6e4), ("bf16", -1.0, -4.5e4, -3.3e4), ("bf16", 0.125, 6e9, 4e9), ("bf16", 0.125, 2e9, -7e8)])
@pytest.mark.parametrize("shape", SHAPES)
def test_scores_far_from_zero(shape, dtype, scale, a, b):
    """Scores so large that their product with the scale is off by more than the exponents of the
    types span."""
    note(f"scores {scale} * {a} * {b} {dtype} {shape}")
    check_equal_scores(equal_scores(dtype, shape, a, b), scale, a, b)


@pytest.mark.parametrize("scale,a,b", [(0.125, 2.0 ** 60, -(2.0 ** 57)), (1.0, 3e18, -1e19), (-1.0, -3e18, -3e19)])
@pytest.mark.parametrize("shape", SHAPES)
def test_scores_near_the_lowest_number(shape, scale, a, b):
    """Rows all of whose scores lie far below any that a mask stands for."""
    note(f"scores {scale} * {a} * {b} {shape}")
    check_equal_scores(equal_scores("bf16", shape, a, b), scale, a, b)


@pytest.mark.parametrize("scale", [1e9, 1e30])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("shape", SHAPES)
def test_large_scales_of_small_scores(shape, window, scale):
    """A scale that, times the reference of a row that has seen nothing yet, passes fp32: such rows
    begin inside a tile of keys that the window or the chunk's order hides."""
    note(f"scale {scale} window={window} {shape}")
    c = make_case(7, *([shape[0], (4, 2), 64, 16, "bf16", shape[1]]))
    c.q.div_(scale ** 0.5), c.k.div_(scale ** 0.5)
    out, lse = run(c, window, 0, scale)
    scale = float(np.float32(scale))
    check(out, lse, reference(c, scale, window, 0), c, scale, "large scale")


# ----------------------------------------------------------------------------- small scales

@pytest.mark.parametrize("scale", [0.0, 1e-31, -1e-38, 1e-12])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_scales_at_and_near_zero(shape, dtype, scale):
    """Every seen value weighs the same: their mean, and the logarithm of their number."""
    note(f"scale {scale} {dtype} {shape}")
    c = make_case(9, shape[0], (4, 2), 64, 16, dtype, shape[1])
    for window, sinks in ((0, 0), (100, 3)):
        out, lse = run(c, window, sinks, scale)
        ref = reference(c, scale, window, sinks)
        count = ref[-1]
        assert np.allclose(ref[1], np.where(count > 0, np.log(np.maximum(count, 1)), -np.inf)[:, None], atol=1e-9)
        check(out, lse, ref, c, scale, f"scale {scale} window={window}")


# ------------------------------------------------------------- values that are not finite

INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("length,n,heads,window", [
    (200, 100, (4, 4), 0), (200, 100, (8, 2), 40),          # one group of waves
    (1300, 150, (2, 2), 0), (1300, 150, (2, 2), 513),       # two groups
    (4001, 128, (2, 2), 0), (4001, 128, (2, 2), 2000),      # blocks cut into parts
    (300, 1, (4, 2), 0), (2900, 1, (2, 1), 0), (2900, 1, (2, 1), 700)])
def test_values_that_are_not_finite_stay_in_their_dims(length, n, heads, window, dim, dtype):
    """Finite keys; single dims of single values are infinite or no number, in tiles that some rows
    see in part (the chunk's own tokens, the window's first ones) and in ones that all see.  Rows
    that see one have in that dim the infinity (two of both signs, or no number: no number); every
    other dim, and the rows that do not see it, are as without."""
    past = length - n
    first = max(0, past - window + 1) if window else 0      # of what the first row sees
    plants = [(length - 1, 3, INF), (past + n // 2, 4, -INF), (past + n // 3, 5, INF), (past + n // 4, 5, -INF),
              (past + n // 5, 6, NAN), (first + 1, 33, -INF), (first + n // 2, 34, NAN), (first + n // 2, 35, INF),
              (first + 2 * n // 3, 36, INF), (first + n // 2 + 1, 36, -INF), ((first + past) // 2, 62, INF),
              (past - 1, 63, -INF), (1, 11, INF), (2, 12, NAN)]
    plants = [(j, d, x) for (j, d), x in {(j, d): x for j, d, x in plants}.items()]
    sinks = 2 if window else 0
    c = make_case(length, [length], heads, dim, 16, dtype, None if n == 1 else [n], gain=0.7)
    scale = 1 / math.sqrt(dim)
    clean = reference(c, scale, window, sinks)
    for j, d, x in plants:
        c.v[c.table[0, j // 16], :, j % 16, d] = x
    note(f"not finite: length={length} n={n} window={window} dim={dim} {dtype}")
    out, lse = run(c, window, sinks)
    got, p = f64(out), past + np.arange(n)
    sees = [(j <= p) & ((p - j < window) | (j < sinks) if window else True) for j, _, _ in plants]
    want = np.zeros((n, dim))                               # 0: as without
    for rows, (_, d, x) in zip(sees, plants):
        with np.errstate(invalid="ignore"):
            want[rows, d] += x                              # inf - inf, as inf + NaN, is NaN
    for h in range(heads[0]):
        for x in (INF, -INF):
            assert (got[:, h][want == x] == x).all(), (h, x)
        assert np.isnan(got[:, h][np.isnan(want)]).all(), h
    planted = np.broadcast_to((want != 0)[:, None], got.shape)
    assert planted.any()
    # the others against the oracle without the plants (whose own dims are left out on both sides)
    fixed = out.clone()
    fixed[torch.from_numpy(planted.copy()).cuda()] = torch.from_numpy(clean[0][planted]).to(out.dtype).cuda()
    check(fixed, lse, clean, c, scale, "the other dims")


# ---------------------------------------------------------------------- q_starts past the rows

@pytest.mark.parametrize("starts", [[0, 8, 30], [-4, 8, 20], [0, 8, 2 ** 31 - 1], [-(2 ** 31), 8, 2 ** 31 - 1], [0, 25, 40]])
def test_append_and_chunks_agree_on_rows_where_q_starts_leave_them(starts):
    """q_starts count as 0 below it and as the number of rows above it, for both calls: keys and
    values land where the queries of the same rows look for them."""
    note(f"append and chunk, q_starts={starts}")
    T, lens = 20, [25, 60]
    c = make_case(5, lens, (4, 2), 64, 16, "f16", [8, 12])
    gen = torch.Generator().manual_seed(3)
    new = [torch.randn((T, 2, 64), generator=gen).half() for _ in range(2)]
    k, v = c.k.cuda(), c.v.cuda()
    cache = attn.SpearKVCache(k, v)
    batch = attn.SpearKVBatch(on_gpu(c.table), on_gpu(lens), on_gpu(starts))
    bounded = [min(max(s, 0), T) for s in starts]
    attn.spear_kv_append(cache, batch, new[0].cuda(), new[1].cuda())
    want = [torch.from_numpy(attn_ref.append_ref(old.numpy(), x.numpy(), c.table, lens, bounded))
            for old, x in ((c.k, new[0]), (c.v, new[1]))]
    assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])
    ws = attn.new_attn_workspace(cache, 4, 2, T)
    out, lse = attn.spear_attn_prefill(cache, batch, c.q.cuda(), workspace=ws, return_lse=True)
    c = Case(c.q, *want, c.table, lens, bounded, "f16")
    check(out, lse, reference(c, 1 / 8, 0, 0), c, 1 / 8, "the chunk after it")


def test_append_of_more_pieces_than_a_launch_has_threads():
    """2^24 tokens of 32 heads are 2^32 pieces of 16 bytes; all but three pages' tokens are dropped."""
    note("append of 2^24 tokens")
    n, page = 1 << 24, 16
    k, v = (torch.zeros((4, 32, page, 64), dtype=torch.float16, device="cuda") for _ in range(2))
    table = torch.full((1, n // page), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, n // page // 2], table[0, -1] = 2, 0, 1
    batch = attn.SpearKVBatch(table, on_gpu([n]), on_gpu([0, n]))
    new = torch.arange(1, 1 + 2 * 32 * 64, dtype=torch.float32, device="cuda").div(4096).half().view(2, 1, 32, 64)
    attn.spear_kv_append(attn.SpearKVCache(k, v), batch, new[0].expand(n, 32, 64), new[1].expand(n, 32, 64))
    for t, x in ((k, new[0, 0]), (v, new[1, 0])):
        for p in (0, 1, 2):
            assert torch.equal(t[p], x[:, None].expand(32, page, 64)), p
        assert not t[3].any()
