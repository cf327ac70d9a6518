"""One attention block served with libspear: compensated 4-bit projections, a paged cache, chunked
prompts, forked samples.

    python examples/serve_block.py

A block is a fused query-key-value projection and an output projection (SpearLayer), with attention
over the paged cache between them.  The script serves two prompts in chunks (both in one batch),
forks each into samples that share the prompt's pages, decodes a few tokens of all of them in one
batch a step, ends some, compacts the pool and goes on.  Random weights and inputs.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_gemm_error_amd import attn, spear, synth  # noqa: E402


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Block:
    """The projections and the cache of one layer."""

    def __init__(self, hidden=1024, q_heads=16, kv_heads=4, head_dim=64, pages=256, page_size=16, slots=16,
                 max_len=1024, rank=16, window=0, sinks=0, seed=1):
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.window, self.sinks = window, sinks
        wide = (q_heads + 2 * kv_heads) * head_dim
        self.qkv = spear.layer_to_device(synth.make_layer(wide, hidden, 128, rank, seed=seed))
        self.out = spear.layer_to_device(synth.make_layer(hidden, q_heads * head_dim, 128, rank, seed=seed + 1))
        k, v = (torch.zeros((1, pages, kv_heads, page_size, head_dim), dtype=torch.float16, device="cuda")
                for _ in range(2))
        self.all_layers = attn.SpearKVCache(k, v)      # for the page calls
        self.cache = self.all_layers.layer(0)          # for append and attention
        self.pool = attn.SpearKVPool.new(pages, page_size, slots, -(-max_len // page_size))
        self.linear_ws = {}
        self.attn_ws = attn.new_attn_workspace(self.cache, q_heads, slots, 4096)

    def _linear(self, layer, x):
        ws = self.linear_ws.get(id(layer))
        if ws is None or spear.spear_workspace_bytes(layer, x.shape[0]) > ws.numel():
            ws = self.linear_ws[id(layer)] = spear.new_workspace(layer, x.shape[0])
        return spear.spear_linear(layer, x, workspace=ws)

    def step(self, x, slots, lens, rows=None):
        """New tokens x [tokens][hidden] of the sequences in `slots`, whose lengths become `lens`;
        rows: the first row of each and the end (None: one row each) -> the block's output."""
        missing = attn.spear_kv_reserve(self.pool, self.all_layers, slots, lens)
        batch = attn.SpearKVBatch(self.pool.table[slots.long()], lens, rows)
        heads = self._linear(self.qkv, x).unflatten(1, (-1, self.head_dim))
        q = heads[:, :self.q_heads]
        k = heads[:, self.q_heads:self.q_heads + self.kv_heads]
        v = heads[:, self.q_heads + self.kv_heads:]
        attn.spear_kv_append(self.cache, batch, k, v)
        call = attn.spear_attn_decode if rows is None else attn.spear_attn_prefill
        o = call(self.cache, batch, q, window=self.window, sinks=self.sinks, workspace=self.attn_ws)
        return self._linear(self.out, o.flatten(1)), missing


def serve(block, prompts=(300, 217), chunk=128, samples=3, tokens=8, compact_at=4, seed=0):
    """-> the outputs of the decode steps, [step] of [sequences still running][hidden]."""
    hidden = block.qkv.K
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = [torch.randn((n, hidden), generator=gen, device="cuda").half() for n in prompts]
    done = [0] * len(prompts)
    while any(d < n for d, n in zip(done, prompts)):
        now = [min(chunk, n - d) for d, n in zip(done, prompts)]
        live = [i for i, n in enumerate(now) if n]
        rows = [0]
        for i in live:
            rows.append(rows[-1] + now[i])
        xs = torch.cat([x[i][done[i]:done[i] + now[i]] for i in live])
        done = [d + n for d, n in zip(done, now)]
        _, missing = block.step(xs, _ints(live), _ints([done[i] for i in live]), _ints(rows))
        assert int(missing) == 0, "the pool is too small"
    # every prompt's samples share its pages; the first one goes on in the prompt's own slot
    P = len(prompts)
    src = [i for i in range(P) for _ in range(samples - 1)]
    dst = list(range(P, P + len(src)))
    attn.spear_kv_fork(block.pool, _ints(src), _ints(dst))
    slots, lens = list(range(P)) + dst, list(prompts) + [prompts[i] for i in src]
    outputs = []
    for t in range(tokens):
        if t == compact_at:  # the last sample of each prompt ends
            gone = [s for j, s in enumerate(dst) if j % (samples - 1) == samples - 2]
            attn.spear_kv_free(block.pool, _ints(gone))
            lens = [n for n, s in zip(lens, slots) if s not in gone]
            slots = [s for s in slots if s not in gone]
            attn.spear_kv_compact(block.pool, block.all_layers)
        lens = [n + 1 for n in lens]
        xt = torch.randn((P + len(dst), hidden), generator=gen, device="cuda").half()[slots]
        y, missing = block.step(xt, _ints(slots), _ints(lens))
        assert int(missing) == 0, "the pool is too small"
        outputs.append(y)
    return outputs


def main():
    torch.cuda.set_device(0)
    block = Block()
    for i, y in enumerate(serve(block)):
        print(f"decode step {i}: {y.shape[0]} sequences, rms {y.float().square().mean().sqrt().item():.4f}")
    used = int((block.pool.refs > 0).sum())
    print(f"{used} of {block.pool.refs.numel()} pages in use, the highest {int((block.pool.refs > 0).nonzero().max())}")


if __name__ == "__main__":
    main()
