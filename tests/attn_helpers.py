"""Cases and tolerances of the attention and cache tests (not a test module)."""

from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

from oracle import attn_ref

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@dataclass
class Case:
    """Host tensors of one step: k, v [pages][heads][page][dim], q [tokens][heads][dim]."""

    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    table: np.ndarray
    lens: list
    starts: list | None
    dtype: str


def make_case(seed, lens, heads, dim, page, dtype="f16", chunks=None, spare=3, unused=None, gain=1.5):
    """Random pages in random order; `chunks`: new tokens per sequence (None: one each); `unused`:
    what cache slots hold that belong to no token (default: random values)."""
    gen = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    Hq, Hkv = heads
    rows = [-(-n // page) for n in lens]
    P, W = sum(rows) + spare, max(1, max(rows, default=1)) + 1
    order = rng.permutation(P)
    table = np.full((len(lens), W), -1, dtype=np.int32)
    at = 0
    for b, r in enumerate(rows):
        table[b, :r] = order[at:at + r]
        at += r
    dt = DTYPES[dtype]
    k = torch.randn((P, Hkv, page, dim), generator=gen).to(dt)
    v = torch.randn((P, Hkv, page, dim), generator=gen).to(dt)
    if unused is not None:
        free = torch.ones((P, page), dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(n):
                free[table[b, j // page], j % page] = False
        for t in (k, v):
            t.transpose(1, 2)[free] = unused
    starts = None if chunks is None else [0] + [int(x) for x in np.cumsum(chunks)]
    T = len(lens) if chunks is None else starts[-1]
    q = (gain * torch.randn((T, Hq, dim), generator=gen)).to(dt)
    return Case(q, k, v, table, list(lens), starts, dtype)


def as_layout(t, layout):
    """The pages [..., heads, page, dim] on the GPU in another memory order, the same shape."""
    t = t.cuda()
    if layout == "head":
        return t.contiguous()
    if layout == "token":
        return t.transpose(-3, -2).contiguous().transpose(-3, -2)
    # inside a larger array: two planes per page, rows of dim + 8 elements
    big = torch.full((*t.shape[:-3], 2, *t.shape[-3:-1], t.shape[-1] + 8), float("nan"),
                     dtype=t.dtype, device="cuda")
    view = big[..., 1, :, :, :t.shape[-1]]
    view.copy_(t)
    return view


def on_gpu(v):
    return None if v is None else torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().cpu().double().numpy()


def reference(c: Case, scale, window, sinks):
    """The oracle on the case; hidden values that are not finite are kept out of its products."""
    return attn_ref.attention_ref(f64(c.q), f64(c.k), f64(c.v), c.table, c.lens, c.starts, scale,
                                  window, sinks)


def check(out, lse, ref, c: Case, scale, what=""):
    """Elementwise against the oracle.  With h = eps / 2 of the type: the softmax weights are
    rounded once to the type before they meet the values (h times sum p |v| / l; in fp16 also
    2^-25 absolute below its normal range, 2^-25 sum |v| / l), the result once (h |o|, half the
    smallest subnormal in fp16).  A score is a sum of D fp32 products and changes by at most
    (D + 4) 2^-24 reach, and a weight by as much relatively, twice as l has it too; exponent and
    sums add 2^-20 and count 2^-24."""
    o_ref, lse_ref, spread, vsum, reach, count = ref
    D = c.q.shape[-1]
    h = torch.finfo(DTYPES[c.dtype]).eps / 2
    tiny = 2.0 ** -25 if c.dtype == "f16" else 0.0
    score = (D + 4) * 2.0 ** -24 * reach
    fp32 = 2 * score + 2.0 ** -20 + count[:, None] * 2.0 ** -24
    tol = h * (spread + np.abs(o_ref)) + tiny * (vsum + 1) + (1 + h) * fp32[..., None] * spread
    got = f64(out)
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = float(np.max(np.abs(got - o_ref) - tol, initial=-1.0))
    at = np.unravel_index(np.argmax(np.abs(got - o_ref) - tol), got.shape) if got.size else None
    assert worst <= 0, f"{what}: out at {at}: {got[at]} for {o_ref[at]}, tolerance {tol[at]}"
    if lse is None:
        return
    z = f64(lse)
    empty = np.isneginf(lse_ref)
    assert np.array_equal(np.isneginf(z), empty), f"{what}: rows that see nothing"
    ztol = score + 2.0 ** -20 + (count[:, None] + 8) * 2.0 ** -24 + 2.0 ** -21 * np.where(empty, 0, np.abs(lse_ref))
    assert (np.abs(z[~empty] - lse_ref[~empty]) <= ztol[~empty]).all(), f"{what}: lse"
