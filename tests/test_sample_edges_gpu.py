"""Sampling where it can go wrong beside test_sample_gpu.py's cases: tokens that lie on a bin's border
but for the rounding of their depth, and draws at the end of what is kept."""

import numpy as np
import pytest

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
