"""The microscaled, norm and sampling entry points without a GPU: the exports, the C ABI's refusals
(before any launch), sizes, and the binding's checks on CPU tensors."""

import ctypes
import os
import re

import pytest

from quantized_gemm_error_amd import mx, sampling, spear

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
A = ctypes.addressof


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(spear.LIB_PATH):
        pytest.fail("libspear.so is not built: run python -m quantized_gemm_error_amd.build")
    sampling.load_library()
    return mx.load_library()


@pytest.mark.parametrize("header,module", [("spear_mx.h", mx), ("spear_sample.h", sampling)])
def test_exports_every_declared_function(lib, header, module):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    declared = set(re.findall(r"\b(spear_[a-z0-9_]+)\s*\(", text))
    assert declared == set(module.EXPORTED)
    for name in declared:
        assert hasattr(lib, name), name


def _struct(cls, base, kw):
    f = dict(base, **kw)
    return cls(*[f[n] for n, _ in cls._fields_])


def _mx(**kw):
    return _struct(mx.SpearMXC, dict(format=0, rows=64, cols=256, codes=1 << 32, scales=1 << 33), kw)


BAD_MATRICES = [
    (dict(format=2), INVALID), (dict(format=-1), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
    (dict(rows=(1 << 24) + 1), UNSUPPORTED), (dict(cols=(1 << 20) + 1), UNSUPPORTED),
    (dict(rows=1 << 24, cols=1 << 20), UNSUPPORTED), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(codes=(1 << 32) + 128), INVALID), (dict(scales=(1 << 32) + 16), INVALID),
]


@pytest.mark.parametrize("kw,status", BAD_MATRICES)
def test_matrix_refusals(lib, kw, status):
    m = _mx(**kw)
    assert lib.spear_mx_quantize(1 << 34, 0, 256, A(m), None) == status
    assert lib.spear_mx_dequantize(A(m), 1 << 34, 0, 1 << 21, None) == status
    args = _linear(w=A(m))
    assert lib.spear_mx_linear(A(args), 1 << 40, 1 << 40, None) == status
    assert spear.spear_last_error()


def test_quantize_and_dequantize_refusals(lib):
    m = _mx()
    assert lib.spear_mx_quantize(1 << 34, 0, 256, None, None) == INVALID
    for x, dtype, stride in ((None, 0, 256), (1 << 34, 3, 256), (1 << 34, -1, 256), (1 << 34, 0, -8),
                             ((1 << 34) + 1, 0, 256), ((1 << 34) + 2, 2, 256), (1 << 34, 0, 1 << 41)):
        assert lib.spear_mx_quantize(x, dtype, stride, A(m), None) == INVALID
    for out, dtype, stride in ((None, 0, 256), (1 << 34, 3, 256), (1 << 34, 0, 255), ((1 << 34) + 2, 2, 256)):
        assert lib.spear_mx_dequantize(A(m), out, dtype, stride, None) == INVALID
    empty = _mx(rows=0, codes=None, scales=None)
    assert lib.spear_mx_quantize(None, 0, 256, A(empty), None) == 0
    assert lib.spear_mx_dequantize(A(empty), None, 0, 256, None) == 0


def _norm(**kw):
    return _struct(mx.SpearNormArgsC, dict(
        dtype=0, rows=64, hidden=256, x=1 << 32, residual=1 << 33, weight=1 << 34, x_stride=256, residual_stride=256,
        residual_out=1 << 35, out=1 << 36, residual_out_stride=256, out_stride=256, out_mx=None, eps=1e-5), kw)


BAD_NORMS = [
    (dict(dtype=2), INVALID), (dict(rows=-1), INVALID), (dict(hidden=0), INVALID), (dict(hidden=65537), UNSUPPORTED),
    (dict(rows=(1 << 24) + 1), UNSUPPORTED), (dict(eps=-1e-9), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(out=None), INVALID), (dict(x=None), INVALID), (dict(weight=None), INVALID),
    (dict(residual=None), INVALID), (dict(residual_out=None), INVALID), (dict(x=(1 << 32) + 1), INVALID),
    (dict(x_stride=-1), INVALID), (dict(out_stride=255), INVALID), (dict(residual_out_stride=0), INVALID),
    (dict(out=1 << 35), INVALID), (dict(out=1 << 32, out_stride=264), INVALID),
    (dict(residual_out=1 << 33, residual_stride=0), INVALID),
]


@pytest.mark.parametrize("kw,status", BAD_NORMS)
def test_norm_refusals(lib, kw, status):
    assert lib.spear_rms_norm(A(_norm(**kw)), None) == status


def test_norm_into_a_matrix(lib):
    m = _mx()
    assert lib.spear_rms_norm(A(_norm(out_mx=A(m))), None) == INVALID          # two outputs
    for kw in (dict(rows=63), dict(cols=255), dict(format=5), dict(codes=None)):
        m = _mx(**kw)
        assert lib.spear_rms_norm(A(_norm(out=None, out_mx=A(m))), None) == INVALID
    m = _mx(rows=0, codes=None, scales=None)
    assert lib.spear_rms_norm(A(_norm(rows=0, out=None, out_mx=A(m))), None) == 0
    assert lib.spear_rms_norm(A(_norm(rows=0)), None) == 0
    assert lib.spear_rms_norm(None, None) == INVALID


_W = _mx()


def _linear(**kw):
    return _struct(mx.SpearMXLinearArgsC, dict(
        w=A(_W), x_mx=None, x=1 << 35, x_dtype=0, x_format=1, n_tokens=3, x_stride=256, y=1 << 36, y_dtype=0,
        y_stride=64), kw)


BAD_LINEARS = [
    (dict(w=None), INVALID), (dict(x=None), INVALID), (dict(x_mx=A(_W)), INVALID), (dict(x_dtype=2), INVALID),
    (dict(x_format=2), INVALID), (dict(n_tokens=-1), INVALID), (dict(x_stride=-1), INVALID), (dict(y=None), INVALID),
    (dict(y_dtype=3), INVALID), (dict(y_stride=63), INVALID), (dict(n_tokens=(1 << 24) + 1), UNSUPPORTED),
    (dict(x=(1 << 35) + 1), INVALID), (dict(y=(1 << 36) + 2, y_dtype=2), INVALID),
]


@pytest.mark.parametrize("kw,status", BAD_LINEARS)
def test_linear_refusals(lib, kw, status):
    assert lib.spear_mx_linear(A(_linear(**kw)), 1 << 40, 1 << 40, None) == status


def test_linear_operands_and_workspace(lib):
    eight = _mx(format=1)
    assert lib.spear_mx_linear(A(_linear(w=A(eight))), 1 << 40, 1 << 40, None) == UNSUPPORTED
    short = _mx(cols=128)
    assert lib.spear_mx_linear(A(_linear(x=None, x_mx=A(short))), 1 << 40, 1 << 40, None) == INVALID
    need = lib.spear_mx_workspace_bytes(A(_W), 3)
    assert need >= lib.spear_mx_code_bytes(1, 3, 256) + lib.spear_mx_scale_bytes(1, 3, 256)
    for ws, n in ((None, need), (1 << 40, need - 1), ((1 << 40) + 64, need)):
        assert lib.spear_mx_linear(A(_linear()), ws, n, None) == WORKSPACE
    assert lib.spear_mx_linear(A(_linear(n_tokens=0)), None, 0, None) == 0
    assert lib.spear_mx_linear(A(_linear(n_tokens=0, x=None, y=None)), None, 0, None) == 0
    none = _mx(rows=0, codes=None, scales=None)
    assert lib.spear_mx_linear(A(_linear(w=A(none), y_stride=0)), None, 0, None) == 0


def _sample(**kw):
    return _struct(sampling.SpearSampleArgsC, dict(
        logits=1 << 32, dtype=2, rows=4, vocab=1000, stride=1000, u=1 << 33, temperature=None, top_k=None, top_p=None,
        min_p=None, tokens=1 << 34, logprobs=None), kw)


BAD_SAMPLES = [
    (dict(dtype=3), INVALID), (dict(rows=-1), INVALID), (dict(vocab=0), INVALID), (dict(vocab=(1 << 18) + 1), UNSUPPORTED),
    (dict(rows=(1 << 20) + 1), UNSUPPORTED), (dict(logits=None), INVALID), (dict(logits=(1 << 32) + 2), INVALID),
    (dict(stride=-1), INVALID), (dict(u=None), INVALID), (dict(tokens=None), INVALID), (dict(u=(1 << 33) + 2), INVALID),
    (dict(top_k=(1 << 33) + 1), INVALID), (dict(logprobs=(1 << 33) + 2), INVALID),
]


@pytest.mark.parametrize("kw,status", BAD_SAMPLES)
def test_sample_refusals(lib, kw, status):
    assert lib.spear_sample(A(_sample(**kw)), 1 << 40, 1 << 40, None) == status


def test_sample_workspace(lib):
    need = lib.spear_sample_workspace_bytes(4, 1000)
    assert need >= sampling.SPEAR_SAMPLE_HEADER_BYTES
    for ws, n in ((None, need), (1 << 40, need - 1), ((1 << 40) + 64, need)):
        assert lib.spear_sample(A(_sample()), ws, n, None) == WORKSPACE
    assert lib.spear_sample(A(_sample(rows=0)), None, 0, None) == 0
    assert lib.spear_sample(None, None, 0, None) == INVALID
    for rows, vocab in ((-1, 5), (1, 0), (1, (1 << 18) + 1), ((1 << 20) + 1, 5)):
        assert lib.spear_sample_workspace_bytes(rows, vocab) == 0
    assert sampling.spear_sample_workspace_bytes(2 ** 40, 5) == 0
    assert sampling.spear_sample_workspace_bytes(5, 2 ** 32 + 5) == 0


def test_sizes_grow_with_their_arguments(lib):
    for fmt, tile in ((0, 1024), (1, 2048)):
        for rows, cols in ((1, 1), (16, 128), (17, 129), (100, 513), (4096, 11008)):
            rb, kt, kq = -(-rows // 16), -(-cols // 128), -(-cols // 512)
            assert lib.spear_mx_code_bytes(fmt, rows, cols) == rb * kt * tile
            assert lib.spear_mx_scale_bytes(fmt, rows, cols) == rb * kq * 256
            assert mx._mx_bytes(fmt, rows, cols) == (rb * kt * tile, rb * kq * 256)
    assert lib.spear_mx_code_bytes(1, 1 << 24, 1 << 20) == (1 << 20) * (1 << 13) * 2048
    for bad in ((2, 4, 4), (0, -1, 4), (0, 4, 0), (0, (1 << 24) + 1, 4)):
        assert lib.spear_mx_code_bytes(*bad) == 0 and lib.spear_mx_scale_bytes(*bad) == 0
    last = 0
    for n in range(1, 600):
        now = lib.spear_mx_workspace_bytes(A(_W), n)
        assert now >= last
        last = now
    assert lib.spear_mx_workspace_bytes(A(_W), -1) == 0 and lib.spear_mx_workspace_bytes(None, 4) == 0
    last = 0
    for rows in (1, 2, 3, 7, 8, 31, 64, 100, 255, 256, 257, 1000):
        now = lib.spear_sample_workspace_bytes(rows, 50000)
        assert now >= last
        last = now


def test_binding_checks():
    x = torch.zeros((4, 64), dtype=torch.float16)
    w = torch.zeros(64, dtype=torch.float16)
    for call in (lambda: mx.spear_mx_quantize(x, "fp4"), lambda: mx.spear_rms_norm(x, w),
                 lambda: mx.spear_rms_norm(x, w, out_format="fp8"),
                 lambda: sampling.spear_sample(x, torch.zeros(4)),
                 lambda: mx.spear_mx_linear(mx.SpearMX.empty(8, 64, "fp4", "cpu"), x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for bad in ("int4", None, 7, [1]):
        with pytest.raises(ValueError, match="format"):
            mx.SpearMX.empty(4, 64, bad, "cpu")
    with pytest.raises(spear.SpearError):
        mx.SpearMX.empty(4, 0, "fp4", "cpu")
    with pytest.raises(ValueError, match="32 bits"):
        mx.SpearMX.empty(2 ** 32 + 4, 64, "fp4", "cpu")
    m = mx.SpearMX.empty(4, 64, "fp4", "cpu")
    with pytest.raises(ValueError):
        mx.SpearMX(m.codes[:-1], m.scales, 4, 64, "fp4")
    with pytest.raises(TypeError):
        mx.SpearMX(m.codes.view(torch.int8), m.scales, 4, 64, "fp4")
    with pytest.raises(TypeError):
        mx.spear_mx_quantize(x.double())
    with pytest.raises(ValueError, match="contiguous"):
        mx.spear_mx_quantize(x.t())
    with pytest.raises(ValueError):
        mx.spear_mx_quantize(x, out=mx.SpearMX.empty(5, 64, "fp4", "cpu"))
    with pytest.raises(TypeError):
        mx.spear_rms_norm(x.float(), w.float())
    with pytest.raises(TypeError):
        mx.spear_rms_norm(x, w.bfloat16())
    with pytest.raises(ValueError):
        mx.spear_rms_norm(x, w[:-1])
    with pytest.raises(ValueError):
        mx.spear_rms_norm(x, w, residual_out=x.clone())
    with pytest.raises(ValueError, match="overlaps"):
        big = torch.zeros((5, 64), dtype=torch.float16)
        mx.spear_rms_norm(big[:4], w, out=big[1:])
    with pytest.raises(ValueError, match="overlaps"):
        mx.spear_rms_norm(x, w, residual=x.clone(), residual_out=x, out=x)
    with pytest.raises(ValueError):
        mx.spear_rms_norm(x, w, out=mx.SpearMX.empty(4, 64, "fp4", "cpu"), out_format="fp8")
    with pytest.raises(ValueError, match="columns"):
        mx.spear_mx_linear(mx.SpearMX.empty(8, 32, "fp4", "cpu"), x)
    with pytest.raises(ValueError):
        mx.spear_mx_linear(mx.SpearMX.empty(8, 64, "fp4", "cpu"), x, y=x[:, :7])
    with pytest.raises(TypeError):
        sampling.spear_sample(x, torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError):
        sampling.spear_sample(x, torch.zeros(3))
    with pytest.raises(TypeError):
        sampling.spear_sample(x, torch.zeros(4), top_k=torch.zeros(4))
    with pytest.raises(ValueError, match="overlap"):
        u = torch.zeros(4)
        sampling.spear_sample(x, u, tokens=u.view(torch.int32))
