"""Sampling where it can go wrong beside test_sample_gpu.py's cases: tokens that lie on a bin's border
but for the rounding of their depth, draws at the end of what is kept, and rows and vocabularies that
are counted in several runs, parts or launches."""

import numpy as np
import pytest

from gpu_helpers import note
from oracle import mx_ref
from quantized_gemm_error_amd import sampling
from test_sample_gpu import DT, INF, us, verify

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

# (the largest logit, T): 16 top / T is a whole number, so that 0 is a border between two bins
TOPS = [(1.0, 1.0), (8.0, 1.0), (4.0, 0.5), (12.5, 1.0), (3.0, 2.0), (0.0625, 1.0)]
SMALL = {"1e-20": [1e-20], "-1e-20": [-1e-20], "1e-17": [1e-17], "-1e-17": [-1e-17],
         "normal": [2.0 ** -126, -2.0 ** -126], "subnormal": [2.0 ** -133, -2.0 ** -133],
         "all": [1e-17, -1e-17, 0.0, -0.0, 1e-20, -1e-20, 2.0 ** -126, 2.0 ** -133, -2.0 ** -133, 1e-16, -1e-16]}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("small", list(SMALL))
@pytest.mark.parametrize("top,T", TOPS)
def test_a_bins_border_at_zero(top, T, small, dtype):
    """Logits so small that their depth below the largest rounds onto the border: a list of them
    (up to 2048) and more; alone, and with others above and below."""
    values = torch.tensor(SMALL[small])
    for n in (3, 999, 2047, 2049, 4000):
        rows = 4
        l = torch.full((rows, 5000), -INF)
        gen = torch.Generator().manual_seed(n)
        for r in range(rows):
            at = torch.randperm(5000, generator=gen)
            l[r, at[:n]] = values[torch.randint(0, len(values), (n,), generator=gen)]
            if r >= 2:  # others around
                l[r, at[n:n + 300]] = top * torch.rand(300, generator=gen)
                l[r, at[n + 300:n + 700]] = -T * torch.rand(400, generator=gen)
            l[r, at[-1]] = top
        weight = float(np.exp(-top / T))
        for limits in (dict(), dict(top_k=n // 2 + 1), dict(top_p=0.97), dict(min_p=0.9 * weight),
                       dict(min_p=min(1.0, 1.1 * weight)), dict(top_k=n, top_p=0.9, min_p=0.5 * weight)):
            verify(l.to(DT[dtype]).cuda(), us(n + len(limits), rows), f"border {top} {T} {small} {n} {limits}",
                   temperature=T, **limits)


def test_the_last_token_kept_however_little_it_weighs():
    """u = 1 and above take the last token kept, also where it weighs less than 2^-24 of the others,
    and u below 1 draws up to its own step, 2^-24 from the end.  (Rows of many tokens have u = 1 and
    above only: at 2^-24 from the end their tokens weigh less than the 2e-9 of the row that lie
    within verify()'s distance of a border.)"""
    ends = [1.0, 1.5, INF, 1 - 2.0 ** -24]
    l = torch.tensor([[0.0, -20.0]] * 4)
    tokens, lp = verify(l.cuda(), ends, "two tokens")
    assert tokens.tolist() == [1, 1, 1, 0] and abs(float(lp[0]) + 20) < 1e-5
    assert verify(torch.tensor([[0.0, -63.9, -64.1, -200.0]]).cuda(), [1.0], "e^-64")[0].tolist() == [1]
    gen = torch.Generator().manual_seed(3)
    tail = torch.cat([torch.zeros(3), -20 - 30 * torch.rand(900, generator=gen)])
    tail = tail[torch.randperm(903, generator=gen)].expand(4, 903).contiguous()
    wide = 4 * torch.randn((4, 40000), generator=gen)
    flat = 0.01 * torch.randn((4, 40000), generator=gen)     # thousands of tokens to a bin
    for name, rows in (("tail", tail), ("wide", wide), ("flat", flat), ("equal", torch.full((4, 40000), 2.5))):
        for limits in (dict(), dict(top_k=2), dict(top_k=500), dict(top_k=39999), dict(top_p=0.9), dict(top_p=0.1),
                       dict(top_p=1 - 2.0 ** -24), dict(min_p=1e-9), dict(min_p=0.3), dict(min_p=1.0),
                       dict(top_k=600, top_p=0.95, min_p=1e-4), dict(temperature=0.4), dict(temperature=7.0, min_p=0.01)):
            for dtype in ("f32", "bf16"):
                verify(rows.to(DT[dtype]).cuda(), [1.0, 1.5, INF, 3e38], f"last of {name} {dtype} {limits}", **limits)
    masked = tail.clone()
    masked[:, ::3], masked[1, ::2], masked[2, [5, 9]] = -INF, -INF, INF
    verify(masked.cuda(), [1.0] * 4, "last under a mask")


def test_the_last_token_kept_where_the_limits_bin_has_none():
    """min_p's depth lies in a bin whose tokens are all deeper: the last kept is bins before."""
    for m, depth in ((0.5, 0.7), (1e-3, 6.93), (0.9999, 0.01)):
        l = torch.tensor([[0.0, -0.001 * depth, -depth, -depth - 0.001, -30.0]] * 3)
        for limits in (dict(), dict(top_k=4), dict(top_p=0.999999)):
            verify(l.cuda(), [1.0, 0.99, 0.2], f"none in the limit's bin {m} {limits}", min_p=m, **limits)


def check_rows(logits, rows, what, u, temperature, top_k, top_p, min_p):
    """A call on all rows with limits of their own; the given rows against the oracle (as verify())."""
    note(what)
    n = logits.shape[0]
    ws = sampling.new_sample_workspace(n, logits.shape[1])
    tokens, logprobs = sampling.spear_sample(logits, u, temperature, top_k, top_p, min_p, workspace=ws,
                                             return_logprobs=True)
    torch.cuda.synchronize()
    for r in rows:
        asks = [float(t[r]) for t in (u, temperature, top_k, top_p, min_p)]
        t, lp, kept, near = mx_ref.sample_ref(logits[r].float().cpu().numpy(), asks[0], asks[1], int(asks[2]), *asks[3:])
        assert near > 1e-9 or asks[0] == 0, f"{what} row {r}: the draw is at a border ({near})"
        got, glp = int(tokens[r]), float(logprobs[r])
        assert got == t, f"{what} row {r}: token {got} for {t} of {kept}"
        assert abs(glp - lp) <= 1e-9 + 2.0 ** -24 * abs(lp), f"{what} row {r}: {glp} for {lp}"
    assert (ws[:sampling.SPEAR_SAMPLE_HEADER_BYTES] == 0).all()


def asks_of(n, seed):
    gen = torch.Generator().manual_seed(seed)
    pick = lambda v, t=torch.float32: torch.tensor(v, dtype=t)[torch.randint(0, len(v), (n,), generator=gen)].cuda()  # noqa: E731
    return (torch.rand(n, generator=gen).cuda(), pick([1.0, 1.0, 0.7, 1.5, 0.0]),
            pick([0, 0, 0, 50, 3000], torch.int32), pick([1.0, 1.0, 0.9, 0.5]), pick([0.0, 0.0, 0.01]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab", [(256, 65519), (256, 65520), (256, 65521), (257, 131073), (256, 2 ** 18), (255, 131072),
                                     (200, 2 ** 18), (129, 100003), (128, 2 ** 18 - 1)])
def test_rows_counted_in_several_runs_or_parts(n, vocab, dtype):
    """From 256 rows on one workgroup counts a row in runs of 65520 tokens; fewer rows have as many
    parts at least.  Rows that start at every place of a 16-byte vector; a flat row among them."""
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    pad = 8 * (vocab // 8) + 8 + 3                      # odd: each row starts elsewhere in its vector
    big = (2 * torch.randn((n, pad), generator=gen, device="cuda")).to(DT[dtype])
    l = big[:, 1:1 + vocab]
    l[7] = 0.25
    rows = sorted({0, 1, 2, 3, 7, n // 2, n - 2, n - 1} | set(range(8, n, max(1, n // 8))))
    check_rows(l, rows, f"{n} rows of {vocab} {dtype}", *asks_of(n, vocab + n))


@pytest.mark.parametrize("n", [65535, 65536, 65600, 131075])
def test_more_rows_than_a_grid_holds(n):
    """Rows past the grid's second extent go in launches of their own, each with its arrays' places."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    l = (3 * torch.randn((n, 67), generator=gen, device="cuda")).bfloat16()[:, :65]
    at = {0, 1, 65533, 65534, 65535, 65536, 65537, 131069, 131070, 131071, n - 2, n - 1} | set(range(0, n, n // 60))
    check_rows(l, sorted(r for r in at if r < n), f"{n} rows", *asks_of(n, n))
