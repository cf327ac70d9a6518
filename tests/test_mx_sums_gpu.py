"""What the microscaled products sum in: large products that cancel or meet zeros beside small ones
must leave these their fp32 precision."""

import numpy as np
import pytest

from gpu_helpers import note
from oracle import mx_ref
from quantized_gemm_error_amd import mx

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
MOST = {"fp8": 448.0, "fp4": 6.0}
TOKENS = [1, 4, 16, 33, 64, 65, 300]


def cut(tokens, fmt, out):
    """Whether the calls are those whose products of 8 columns are cut (the header says which)."""
    return tokens > 64 and fmt == "fp8" and out != "f32"


def product(x, w, fmt, out):
    """y by the library and the values that it multiplies, float64."""
    xm, wm = mx.spear_mx_quantize(x.float().cuda(), fmt), mx.spear_mx_quantize(w.float().cuda(), "fp4")
    y = mx.spear_mx_linear(wm, xm, out_dtype=DT[out])
    torch.cuda.synchronize()
    return (y.cpu().double().numpy(), mx_ref.held_ref(x.double().numpy(), fmt), mx_ref.held_ref(w.double().numpy(), "fp4"))


def within(y, ref, reach, K, out, extra, what):
    """Rounded once (eps / 2, or half of fp16's smallest step); before it eight products after eight
    are added, in one step or (e4m3, in two parts) two, and 16 waves' sums join: K / 4 + 16
    roundings of 2^-24 of what is there, at most `reach`, the sum of the products' magnitudes."""
    tol = (K / 4 + 16) * 2.0 ** -24 * reach + extra
    tol = tol + torch.finfo(DT[out]).eps / 2 * (np.abs(ref) + tol) + (2.0 ** -25 if out == "f16" else 0.0)
    worst = np.max(np.abs(y - ref) / np.maximum(tol, 1e-300))
    assert worst <= 1, f"{what}: {worst} of the tolerance"


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("tokens", TOKENS)
def test_small_products_beside_large_ones_that_cancel(tokens, fmt, out):
    """Each row of x holds the largest number twice, with both signs, at columns that go through a
    block of 8 products, and one small number elsewhere in the eight: y is the small product."""
    note(f"cancelling products {tokens} {fmt} {out}")
    K = 256
    x, small = torch.zeros((tokens, K)), [2.0 ** -9, 3 * 2.0 ** -9, 0.0625, 0.40625, 1.75, 2.0, 13.0, 26.0]
    if fmt == "fp4":
        small = [0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 0.5, 1.5]
    for r in range(tokens):
        eight, a, b, c = 8 * (5 * r % 32), r % 8, (r + 1 + r // 8 % 7) % 8, (r + 3) % 8
        if c in (a, b):
            c = next(i for i in range(8) if i not in (a, b))
        x[r, eight + a], x[r, eight + b], x[r, eight + c] = MOST[fmt], -MOST[fmt], small[r % 8]
    w = torch.tensor([6.0, 0.5, 1.5, 3.0])[:, None].expand(4, K).contiguous()
    y, xv, wv = product(x, w, fmt, out)
    ref = xv @ wv.T
    assert (ref != 0).all()
    # the cut: of the eight, one product of at most the largest loses less than a 2^-12th of it
    extra = 2.0 ** -12 * MOST[fmt] * np.abs(wv).max(1)[None] if cut(tokens, fmt, out) else 0.0
    within(y, ref, np.abs(ref), 8, out, extra, f"{tokens} {fmt} {out}")


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", ["zeros", "cancel"])
@pytest.mark.parametrize("tokens", TOKENS)
def test_blocks_of_very_different_scales(tokens, kind, fmt, out):
    """Blocks of a step up to 2^24 apart.  Where the large ones meet zero weights, what the small ones
    make has the precision of these alone.  Where the large ones cancel, a sum in fp32 holds a
    large product until its opposite arrives and is rounded at 2^-24 of it, so the precision is
    that of all products."""
    note(f"far scales {tokens} {kind} {fmt} {out}")
    K, N = 1024, 40
    gen = torch.Generator().manual_seed(tokens)
    x, w = torch.randn((tokens, K), generator=gen), torch.randn((N, K), generator=gen)
    large = torch.rand(K // 32, generator=gen) < 0.4
    power = torch.where(large, torch.randint(4, 25, (K // 32,), generator=gen), torch.zeros(K // 32, dtype=torch.int64))
    x *= torch.exp2(power.float()).repeat_interleave(32)
    cols = large.repeat_interleave(32)
    if kind == "zeros":
        w[:, cols] = 0.0
    else:
        x8, w8 = x.view(tokens, -1, 2, 4), w.view(N, -1, 2, 4)
        at = large.repeat_interleave(4)
        x8[:, at, 1], w8[:, at, 1] = -x8[:, at, 0], w8[:, at, 0]
    y, xv, wv = product(x, w, fmt, out)
    kept = (~cols).numpy()
    ref, reach = xv[:, kept] @ wv[:, kept].T, np.abs(xv) @ np.abs(wv).T
    assert (np.abs(xv @ wv.T - ref) <= 2.0 ** -40 * reach).all()
    extra = 0.0
    if cut(tokens, fmt, out):
        p = np.abs(xv[:, None] * wv[None]).reshape(tokens, N, K // 8, 8)
        extra = (2.0 ** -12 * 8 * p.max(-1) * kept.reshape(-1, 8).all(-1)).sum(-1)
        if kind == "cancel":
            # the cut itself: what a product of a large eight loses, its opposite loses as well or not
            extra = extra + (2.0 ** -12 * 8 * p.max(-1)).sum(-1)
    within(y, ref, reach, K, out, extra, f"{tokens} {kind} {fmt} {out}")
