"""The example block (examples/serve_block.py), the operators as they are used together."""

import os
import sys

import pytest

from gpu_helpers import note

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import serve_block  # noqa: E402

KW = dict(hidden=512, q_heads=8, kv_heads=2, pages=128, slots=8, max_len=512)


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
def test_chunks_forks_and_compaction_change_nothing(window, sinks):
    """The same tokens give the same outputs whatever way the prompt is cut into chunks and
    whenever the pool is compacted: bit for bit where only pages move, and within the rounding of
    the softmax's weights and sums (another order, other reference maxima) for other chunks."""
    note(f"serve block window={window}")
    base = serve_block.serve(serve_block.Block(window=window, sinks=sinks, **KW), compact_at=4)
    block = serve_block.Block(window=window, sinks=sinks, **KW)
    again = serve_block.serve(block, compact_at=4)
    assert all(torch.equal(a, b) for a, b in zip(base, again))
    whole = serve_block.serve(serve_block.Block(window=window, sinks=sinks, **KW), chunk=512, compact_at=4)
    for a, b in zip(base, whole):
        # the cached keys and values come from projections of other row counts: each is a rounded
        # sum of another order, half a step of fp16 (2^-11) off, which a sum of 512 outputs averages
        assert (a.float() - b.float()).norm() <= 2 ** -8 * a.float().norm()


def test_samples_differ_and_share_the_prompt():
    block = serve_block.Block(**KW)
    serve_block.serve(block, tokens=2, compact_at=99)
    refs = block.pool.refs
    assert int(refs.max()) == 3                            # three samples hold the full prompt pages
    held = torch.zeros_like(refs)
    t = block.pool.table
    held.index_add_(0, t[t >= 0].long(), torch.ones_like(t[t >= 0]))
    assert torch.equal(held, refs)
