"""The norm, microscaled matrices and their product beside test_mx_gpu.py's cases: empty batches, matrices
of codes that quantizing does not make."""

import numpy as np
import pytest

from gpu_helpers import note
from oracle import mx_ref
from quantized_gemm_error_amd import mx

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("hidden", [1, 64, 300])
def test_a_norm_of_no_rows(hidden):
    note(f"norm of no rows {hidden}")
    x, res = (torch.zeros((5, hidden), dtype=torch.float16, device="cuda") for _ in range(2))
    w = torch.ones(hidden, dtype=torch.float16, device="cuda")
    for form in (None, "fp4", "fp8"):
        y = mx.spear_rms_norm(x[:0], w, out_format=form)
        y2, h = mx.spear_rms_norm(x[:0], w, residual=res[:0], out_format=form)
        assert tuple(y.shape) == tuple(y2.shape) == tuple(h.shape) == (0, hidden)
    y, h = mx.spear_rms_norm(x[:0], w, residual=res[:0], residual_out=res[:0], out=x[:0])
    assert y.shape == h.shape == (0, hidden)
    m = mx.spear_rms_norm(x[:0], w, out=mx.SpearMX.empty(0, hidden, "fp8"))
    assert mx.spear_mx_dequantize(m).shape == (0, hidden)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_every_code_and_scale_reads_back(fmt):
    """A matrix of a program's own codes: e4m3's code for NaN is NaN, in products too."""
    note(f"every code {fmt}")
    n = 16 if fmt == "fp4" else 256
    codes = np.tile(np.arange(256) % n, (32, 1))[:, :256].astype(np.int64)
    scales = np.tile(np.array([0, 1, 2, 23, 100, 126, 127, 128, 140, 200, 240, 252, 253, 254, 255, 127]), (2, 1))
    scales = np.repeat(scales.reshape(4, 8), 8, axis=0)
    c, s = mx_ref.tiled_ref(codes, scales, fmt)
    m = mx.SpearMX(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), 32, 256, fmt)
    want = mx_ref.values_ref(codes, scales, fmt)
    got = mx.spear_mx_dequantize(m).cpu().double().numpy()
    with np.errstate(over="ignore"):
        assert np.array_equal(got, want.astype(np.float32).astype(np.float64), equal_nan=True)
        for dt in (torch.float16, torch.bfloat16):
            got = mx.spear_mx_dequantize(m, dt).cpu()
            held = torch.from_numpy(want.astype(np.float32)).to(dt)
            assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(held, nan=7.0))
    w = mx.spear_mx_quantize(torch.ones((16, 256), device="cuda"), "fp4")
    y = mx.spear_mx_linear(w, m, out_dtype=torch.float32).cpu().numpy()
    with np.errstate(invalid="ignore"):
        assert np.array_equal(np.isnan(y), np.isnan(want).any(1)[:, None].repeat(16, 1))
