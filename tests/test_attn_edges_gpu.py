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
