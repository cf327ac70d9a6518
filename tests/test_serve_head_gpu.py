"""The example's head (examples/serve_block.py): norm, vocabulary product and draw behind the block's
steps."""

import os
import sys

import numpy as np
import pytest

from gpu_helpers import note
from oracle import mx_ref
from quantized_gemm_error_amd import mx

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import serve_block  # noqa: E402

KW = dict(hidden=512, q_heads=8, kv_heads=2, pages=128, slots=8, max_len=512)


def test_a_head_changes_no_step_and_draws_one_token_each():
    note("serve head")
    base = serve_block.serve(serve_block.Block(**KW))
    runs = [serve_block.serve(serve_block.Block(**KW), head=serve_block.Head(hidden=512)) for _ in range(2)]
    for outputs, drawn in runs:
        assert all(torch.equal(a, b) for a, b in zip(base, outputs))
        for y, (tokens, logprobs) in zip(outputs, drawn):
            assert tokens.shape == logprobs.shape == (y.shape[0],)
            assert ((tokens >= 0) & (tokens < 4000)).all() and (logprobs <= 0).all()
    assert all(torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) for a, b in zip(runs[0][1], runs[1][1]))


def test_logits_and_tokens_are_the_oracles():
    note("serve head oracle")
    head = serve_block.Head(hidden=512, vocab=3001, slots=8)
    gen = torch.Generator().manual_seed(5)
    y, x = torch.randn((7, 512), generator=gen).half(), torch.randn((7, 512), generator=gen).half()
    u = torch.rand(7, generator=gen)
    logits = head.logits(y.cuda(), x.cuda())
    tokens, logprobs = head.tokens(y.cuda(), x.cuda(), u.cuda(), top_p=torch.full((7,), 0.9).cuda())
    h, _ = mx_ref.norm_ref(y.float().numpy(), x.float().numpy(), head.norm.float().cpu().numpy(), 1e-5)
    held = mx_ref.held_ref(h.astype(np.float64), "fp8")
    w = mx.spear_mx_dequantize(head.weight).double().cpu().numpy()
    ref, reach = held @ w.T, np.abs(held) @ np.abs(w).T
    # 512 columns: 4 steps of the product and their join, each at most 2^-23 of what it has reached
    assert (np.abs(logits.double().cpu().numpy() - ref) <= 3 * (4 + 8) * 2.0 ** -23 * reach).all()
    for i in range(7):
        t, lp, _, near = mx_ref.sample_ref(logits[i].cpu().numpy(), float(u[i]), top_p=float(np.float32(0.9)))
        assert near > 1e-9 and int(tokens[i]) == t and abs(float(logprobs[i]) - lp) <= 1e-9 + 2.0 ** -24 * abs(lp)
