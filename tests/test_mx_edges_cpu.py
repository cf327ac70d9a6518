"""Pins of the oracle and refusals beside test_mx_oracle.py's and test_mx_cpu.py's (no GPU)."""

import math

import numpy as np
import pytest

from oracle import mx_ref
from quantized_gemm_error_amd import mx, sampling
from test_mx_cpu import _W, A, INVALID, _linear, _mx, _norm, _sample, lib  # noqa: F401

torch = pytest.importorskip("torch")


def test_the_oracle_draws_the_last_token_kept_from_1_on():
    for u in (1.0, 1.5, math.inf):
        assert mx_ref.sample_ref(np.array([0.0, -20.0]), u)[:2] == (1, pytest.approx(-20.0))
        assert mx_ref.sample_ref(np.array([-63.9, 0.0, -64.1, -200.0]), u)[0] == 0
        assert mx_ref.sample_ref(np.array([0.0, -1.0, -2.0]), u, top_k=2)[0] == 1
        assert mx_ref.sample_ref(np.array([0.0, -1.0, -2.0]), u, min_p=0.5)[0] == 0
    assert mx_ref.sample_ref(np.array([0.0, -20.0]), 1 - 2.0 ** -24)[0] == 0


def test_a_norm_of_no_rows_needs_no_addresses(lib):  # noqa: F811
    for kw in (dict(), dict(residual=None, residual_out=None)):
        assert lib.spear_rms_norm(A(_norm(rows=0, x=None, out=None, **kw)), None) == 0
        assert lib.spear_rms_norm(A(_norm(rows=1, out=None, **kw)), None) == INVALID
    m = _mx(rows=0, codes=None, scales=None)
    assert lib.spear_rms_norm(A(_norm(rows=0, out_mx=A(m))), None) == INVALID   # two outputs


def test_sizes_past_32_bits_are_refused():
    """They would reach the library cut to their low 32 bits."""
    n = 2 ** 32 + 1
    row = torch.zeros((1, 64), dtype=torch.float16)
    tall = row.expand(n, 64)
    w = mx.SpearMX.empty(8, 64, "fp4", "cpu")
    for call in (lambda: mx.spear_rms_norm(tall, row[0]), lambda: mx.spear_rms_norm(tall, row[0], out_format="fp8"),
                 lambda: mx.spear_mx_quantize(tall), lambda: mx.spear_mx_linear(w, tall),
                 lambda: sampling.spear_sample(tall, torch.zeros(1).expand(n))):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_one_row_in_place_whatever_its_stride():
    """A stride between rows says nothing where there is one row (the C ABI takes it so)."""
    big, w = torch.zeros((3, 128), dtype=torch.float16), torch.zeros(64, dtype=torch.float16)
    x = big[:1, :64]
    same = x.as_strided((1, 64), (64, 1))
    for kw in (dict(out=same), dict(residual=same, residual_out=x), dict(residual=x, residual_out=same, out=None)):
        with pytest.raises(ValueError, match="GPU"):   # every check before the device's passes
            mx.spear_rms_norm(x, w, **kw)
    with pytest.raises(ValueError, match="overlaps"):
        mx.spear_rms_norm(big[:2, :64], w, out=big.as_strided((2, 64), (64, 1)))


def test_a_format_that_is_not_outs_is_refused():
    x = torch.zeros((4, 64), dtype=torch.float16)
    for fmt, other in (("fp4", "fp8"), ("fp8", "fp4")):
        m = mx.SpearMX.empty(4, 64, fmt, "cpu")
        with pytest.raises(ValueError, match="another format"):
            mx.spear_mx_quantize(x, other, out=m)
        with pytest.raises(ValueError, match="format"):
            mx.spear_mx_quantize(x, "int4", out=m)
        for given in (fmt, None):
            with pytest.raises(ValueError, match="GPU"):
                mx.spear_mx_quantize(x, given, out=m)
    with pytest.raises(ValueError, match="GPU"):
        mx.spear_mx_quantize(x)


def test_a_workspace_over_an_operand_is_refused(lib):  # noqa: F811
    at, need = 1 << 40, lib.spear_mx_workspace_bytes(A(_W), 3)
    for kw in (dict(x=at + need - 2), dict(x=at - 512 * 2 - 510), dict(y=at), dict(y=at - 2 * 64 * 2 - 126),
               dict(w=_mx(codes=at)), dict(w=_mx(scales=at - 256))):
        held = kw.get("w")
        if held is not None:
            kw = dict(w=A(held))
        assert lib.spear_mx_linear(A(_linear(**kw)), at, need, None) == INVALID, kw
        assert b"workspace" in lib.spear_last_error()
    need = lib.spear_sample_workspace_bytes(4, 1000)
    for kw in (dict(logits=at + need - 4), dict(logits=at - 4 * 4000 + 4), dict(logits=at, stride=0), dict(u=at - 12),
               dict(temperature=at), dict(top_k=at + 64), dict(top_p=at + 4), dict(min_p=at + need - 4),
               dict(tokens=at), dict(logprobs=at - 4)):
        assert lib.spear_sample(A(_sample(**kw)), at, need, None) == INVALID, kw
        assert b"workspace" in lib.spear_last_error()
