"""The example block (examples/serve_block.py), the operators as they are used together."""

import os
import sys

import numpy as np
import pytest

from attn_helpers import Case, check, reference
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


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
def test_outputs_are_the_same_without_compaction(window, sinks, monkeypatch):
    """Bit for bit: compaction moves pages, and nothing that is read from them changes."""
    note(f"serve block with and without compaction, window={window}")
    base = serve_block.serve(serve_block.Block(window=window, sinks=sinks, **KW), compact_at=4)
    held = []
    monkeypatch.setattr(serve_block.attn, "spear_kv_compact", lambda pool, cache: held.append((pool.refs > 0).nonzero()))
    spread = serve_block.serve(serve_block.Block(window=window, sinks=sinks, **KW), compact_at=4)
    assert len(held) == 1 and int(held[0].max()) + 1 > held[0].numel()  # pages that compaction moves
    assert len(base) == len(spread) and all(torch.equal(a, b) for a, b in zip(base, spread))


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
def test_the_blocks_attention_against_the_oracle(window, sinks, monkeypatch):
    """Every step's attention, chunks, forks and compaction on the way, from the keys and values
    that the projections gave for each sequence's own tokens and its parent's."""
    note(f"serve block against the oracle, window={window}")
    block = serve_block.Block(window=window, sinks=sinks, **KW)
    Hq, H, D = block.q_heads, block.kv_heads, block.head_dim
    steps, seen = [], {}
    step, linear, fork = block.step, block._linear, serve_block.attn.spear_kv_fork

    def kept_step(x, slots, lens, rows=None):
        n = slots.numel()
        steps.append({"slots": slots.tolist(), "lens": lens.tolist(),
                      "starts": list(range(n + 1)) if rows is None else rows.tolist()})
        return step(x, slots, lens, rows)

    def kept_linear(layer, x):
        y = linear(layer, x)
        steps[-1]["qkv" if layer is block.qkv else "o"] = (y if layer is block.qkv else x).clone()
        return y

    def kept_fork(pool, src, dst, stream=None):
        steps.append({"fork": list(zip(src.tolist(), dst.tolist()))})
        return fork(pool, src, dst, stream)

    block.step, block._linear = kept_step, kept_linear
    monkeypatch.setattr(serve_block.attn, "spear_kv_fork", kept_fork)
    serve_block.serve(block, tokens=6, compact_at=3)
    torch.cuda.synchronize()
    assert sum("o" in s for s in steps) == 3 + 6           # three steps of chunks, six of single tokens
    for i, s in enumerate(steps):
        if "fork" in s:
            seen.update({b: [t.clone() for t in seen[a]] for a, b in s["fork"]})
            continue
        heads = s["qkv"].cpu().unflatten(1, (-1, D))
        n = len(s["slots"])
        k, v = torch.zeros((2, n, H, max(s["lens"]), D), dtype=heads.dtype)
        for b, slot in enumerate(s["slots"]):
            new = slice(s["starts"][b], s["starts"][b + 1])
            for j, (pages, first) in enumerate(((k, Hq), (v, Hq + H))):
                old = seen.setdefault(slot, [heads.new_zeros((0, H, D)) for _ in range(2)])
                old[j] = torch.cat([old[j], heads[new, first:first + H]])
                assert len(old[j]) == s["lens"][b]
                pages[b, :, :s["lens"][b]] = old[j].transpose(0, 1)
        c = Case(heads[:, :Hq], k, v, np.arange(n)[:, None], s["lens"], s["starts"], "f16")
        check(s["o"].unflatten(1, (Hq, D)), None, reference(c, D ** -0.5, window, sinks), c, D ** -0.5, f"step {i}")
