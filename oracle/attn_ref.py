"""Float64 restatement of the paged cache and its attention (test infrastructure only).

Attention of row i of a sequence's n new tokens, at position p = len - n + i, over the positions j
it sees (j <= p and, with a window w > 0, p - j < w or j < sinks; the page of j must be valid):

    s_j = scale q . k_j,  m = max_j s_j,  l = sum_j e^(s_j - m),
    o = sum_j e^(s_j - m) v_j / l,  lse = m + log l        (nothing seen: o = 0, lse = -inf)

The page bookkeeping is restated entry by entry, as the header describes it.
"""

from __future__ import annotations

import numpy as np


def visible(p: int, n_keys: int, window: int, sinks: int) -> np.ndarray:
    """Boolean [n_keys]: what the query at position p sees."""
    j = np.arange(n_keys)
    see = j <= p
    if window > 0:
        see &= (p - j < window) | (j < sinks)
    return see


def row_pages(table_row, length: int, page_size: int) -> np.ndarray:
    """The page of each of the first `length` positions."""
    return np.asarray(table_row)[np.arange(length) // page_size]


def attention_ref(q, k, v, table, kv_lens, q_starts, scale, window=0, sinks=0):
    """q [T][Hq][D]; k, v [pages][Hkv][page][D] (float64 values); table [B][W]; q_starts None for
    one row per sequence.  -> out [T][Hq][D], lse [T][Hq], spread [T][Hq][D] (sum of p |v| / l, in
    which rounding errors of p show), vsum (sum of |v| / l over what is seen), reach [T][Hq]
    (the largest scale sum |q_d k_d|, in which rounding errors of a score show), count [T]."""
    T, Hq, D = q.shape
    P, Hkv, S, _ = k.shape
    G = Hq // Hkv
    out = np.zeros((T, Hq, D))
    spread, vsum = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    reach = np.zeros((T, Hq))
    count = np.zeros(T, dtype=np.int64)
    starts = list(range(len(kv_lens) + 1)) if q_starts is None else list(q_starts)
    for b, length in enumerate(kv_lens):
        length = max(0, min(int(length), table.shape[1] * S))
        n = starts[b + 1] - starts[b]
        pages = row_pages(table[b], length, S)
        good = (pages >= 0) & (pages < P)
        safe = np.where(good, pages, 0)
        at = np.arange(length) % S
        for i in range(n):
            t, p = starts[b] + i, length - n + i
            see = np.nonzero(visible(p, length, window, sinks) & good)[0]
            count[t] = see.size
            if see.size == 0:
                continue
            for h in range(Hq):
                kk, vv = k[safe[see], h // G, at[see]], v[safe[see], h // G, at[see]]
                s = scale * (kk @ q[t, h])
                m = s.max()
                w = np.exp(s - m)
                l = w.sum()
                out[t, h] = w @ vv / l
                spread[t, h] = w @ np.abs(vv) / l
                vsum[t, h] = np.abs(vv).sum(0) / l
                lse[t, h] = m + np.log(l)
                reach[t, h] = abs(scale) * (np.abs(kk) @ np.abs(q[t, h])).max()
    return out, lse, spread, vsum, reach, count


def append_ref(cache, new, table, kv_lens, q_starts):
    """cache [pages][H][S][D] with the rows of new [T][H][D] stored (a copy)."""
    cache = cache.copy()
    P, _, S, _ = cache.shape
    starts = list(range(len(kv_lens) + 1)) if q_starts is None else list(q_starts)
    for b, length in enumerate(kv_lens):
        length = max(0, min(int(length), table.shape[1] * S))
        n = starts[b + 1] - starts[b]
        for i in range(n):
            p = length - n + i
            if p < 0 or not 0 <= table[b][p // S] < P:
                continue
            cache[table[b][p // S], :, p % S] = new[starts[b] + i]
    return cache


class PoolRef:
    """refs, table, lens (NumPy int32) and the bytes of the pages: pages[p] is any array."""

    def __init__(self, refs, table, lens, page_size, pages):
        self.refs, self.table, self.lens = refs.copy(), table.copy(), lens.copy()
        self.page_size, self.pages = page_size, pages.copy()

    def _row(self, slot, row):
        for c in range(self.table.shape[1]):
            for page, by in ((self.table[slot, c], -1), (row[c], 1)):
                if 0 <= page < len(self.refs):
                    self.refs[page] += by
        self.table[slot] = row

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            if a == b or not (0 <= a < len(self.lens) and 0 <= b < len(self.lens)):
                continue
            self._row(b, self.table[a].copy())
            self.lens[b] = self.lens[a]

    def free(self, slots):
        for s in slots:
            if 0 <= s < len(self.lens):
                self._row(s, np.full(self.table.shape[1], -1, dtype=np.int32))
                self.lens[s] = 0

    def reserve(self, slots, new_lens):
        S, W = self.page_size, self.table.shape[1]
        if any(not 0 <= s < len(self.lens) or n > W * S for s, n in zip(slots, new_lens)):
            return -1
        refs, table, lens, pages = (a.copy() for a in (self.refs, self.table, self.lens, self.pages))
        free = list(np.nonzero(refs == 0)[0])  # pages given up by a copy are not free in this call
        lacking = 0

        def take():
            nonlocal lacking
            if not free:
                lacking += 1
                return -1
            return free.pop(0)

        for s, want in zip(slots, new_lens):
            have = int(lens[s])
            if want <= have:
                continue
            held = -(-have // S)
            last = table[s, held - 1] if have % S else -1
            if last >= 0 and refs[last] > 1:
                page = take()
                if page >= 0:
                    pages[page] = self.pages[last]
                    refs[last] -= 1
                    refs[page] = 1
                    table[s, held - 1] = page
                else:
                    refs[last] -= 1
            for c in range(held, -(-want // S)):
                page = take()
                if page >= 0:
                    table[s, c] = page
                    refs[page] = 1
            lens[s] = want
        if lacking:
            return lacking
        self.refs, self.table, self.lens, self.pages = refs, table, lens, pages
        return 0

    def compact(self):
        used = int((self.refs > 0).sum())
        lo, hi = 0, len(self.refs) - 1
        while True:
            while lo < len(self.refs) and self.refs[lo] > 0:
                lo += 1
            while hi >= 0 and self.refs[hi] <= 0:
                hi -= 1
            if lo >= hi:
                return used
            self.pages[lo] = self.pages[hi]
            self.refs[lo], self.refs[hi] = self.refs[hi], 0
            self.table[self.table == hi] = lo
