"""The norm, microscaled matrices and their product beside test_mx_gpu.py's cases: empty batches."""

import pytest

from gpu_helpers import note
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
