"""Sampling where it can go wrong beside test_sample_gpu.py's cases: tokens that lie on a bin's border
but for the rounding of their depth."""

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
