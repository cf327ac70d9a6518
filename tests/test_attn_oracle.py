"""Pins of the float64 attention and page oracle (CPU): brute force without NumPy on tiny shapes,
closed forms, and the invariants of the page bookkeeping."""

import math

import numpy as np
import pytest

from oracle import attn_ref


def _brute(q, k, v, p, scale, window, sinks):
    seen = [j for j in range(p + 1) if not window or p - j < window or j < sinks]
    if not seen:
        return [0.0] * len(q), -math.inf
    s = [scale * sum(a * b for a, b in zip(q, k[j])) for j in seen]
    z = [math.exp(x) for x in s]
    return [sum(w * v[j][d] for w, j in zip(z, seen)) / sum(z) for d in range(len(q))], math.log(sum(z))


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 3), (3, 0), (3, 1), (4, 9), (1, 0), (100, 5)])
def test_rows_against_brute_force(window, sinks):
    rng = np.random.default_rng(window * 10 + sinks)
    S, D, Hq, Hkv = 2, 3, 4, 2
    lens, starts = [7, 0, 1, 5], [0, 3, 3, 4, 9]
    table = np.array([[3, 1, 7, 0], [-1] * 4, [5, -1, -1, -1], [2, 4, 6, -1]])
    k, v = rng.normal(size=(2, 8, Hkv, S, D))
    q = rng.normal(size=(9, Hq, D))
    out, lse, *_ = attn_ref.attention_ref(q, k, v, table, lens, starts, 0.7, window, sinks)
    for b, n in enumerate(lens):
        rows = starts[b + 1] - starts[b]
        for i in range(rows):
            for h in range(Hq):
                kk = [k[table[b, j // S], h // 2, j % S].tolist() for j in range(n)]
                vv = [v[table[b, j // S], h // 2, j % S].tolist() for j in range(n)]
                o, z = _brute(q[starts[b] + i, h].tolist(), kk, vv, n - rows + i, 0.7, window, sinks)
                assert np.allclose(out[starts[b] + i, h], o, rtol=1e-12, atol=1e-13)
                assert lse[starts[b] + i, h] == pytest.approx(z, rel=1e-12)


def test_equal_keys_average_the_values_and_lse_counts_them():
    v = np.arange(12.0).reshape(3, 1, 4, 1)
    k = np.zeros_like(v)
    out, lse, *_ = attn_ref.attention_ref(np.ones((1, 1, 1)), k, v, np.array([[0, 1, 2]]), [9], None, 1.0, 5, 2)
    seen = [0, 1, 4, 5, 6, 7, 8]
    assert out[0, 0, 0] == pytest.approx(np.mean(seen))
    assert lse[0, 0] == pytest.approx(math.log(len(seen)))


def test_a_page_out_of_range_hides_its_tokens():
    rng = np.random.default_rng(5)
    k, v = rng.normal(size=(2, 3, 1, 2, 4))
    q = rng.normal(size=(1, 1, 4))
    with_hole, *_ = attn_ref.attention_ref(q, k, v, np.array([[0, 9, 2]]), [6], None, 1.0)
    without, *_ = attn_ref.attention_ref(q, k, v, np.array([[0, 2]]), [4], None, 1.0)
    assert np.allclose(with_hole, without)


def test_append_then_read_back():
    cache = np.zeros((4, 1, 2, 1))
    new = np.arange(1.0, 6.0).reshape(5, 1, 1)
    got = attn_ref.append_ref(cache, new, np.array([[2, 0], [1, 3]]), [3, 4], [0, 3, 5])
    assert got[2, 0, :, 0].tolist() == [1, 2] and got[0, 0, :, 0].tolist() == [3, 0]
    assert got[3, 0, :, 0].tolist() == [4, 5] and got[1, 0, :, 0].tolist() == [0, 0]


def _holders(pool):
    n = np.zeros(len(pool.refs), dtype=np.int64)
    for p in pool.table.flatten():
        if p >= 0:
            n[p] += 1
    return n


def test_pool_operations_keep_the_counts_and_the_tokens():
    """Random forks, growth, frees and compactions: refs count the holders, and every slot still
    reads the tokens written to it (token i of slot s carries a tag of its own)."""
    rng = np.random.default_rng(1)
    S, W, slots, P = 4, 6, 7, 60
    pool = attn_ref.PoolRef(np.zeros(P, dtype=np.int32), np.full((slots, W), -1, dtype=np.int32),
                            np.zeros(slots, dtype=np.int32), S, np.zeros((P, S), dtype=np.int64))
    want = {s: [] for s in range(slots)}
    tag = 0
    for step in range(300):
        kind = rng.integers(4)
        if kind == 0:
            a, b = rng.choice(slots, 2, replace=False)
            pool.fork([a], [b])
            want[b] = list(want[a])
        elif kind == 1:
            some = rng.choice(slots, 3, replace=False)
            new = [min(W * S, len(want[s]) + int(rng.integers(0, 6))) for s in some]
            assert pool.reserve(some, new) == 0
            for s, n in zip(some, new):
                while len(want[s]) < n:
                    tag += 1
                    i = len(want[s])
                    assert pool.refs[pool.table[s, i // S]] == 1
                    pool.pages[pool.table[s, i // S], i % S] = tag
                    want[s].append(tag)
        elif kind == 2 and step % 3 == 0:
            s = int(rng.integers(slots))
            pool.free([s])
            want[s] = []
        else:
            used = pool.compact()
            assert (pool.refs[:used] > 0).all() and (pool.refs[used:] == 0).all()
        assert np.array_equal(_holders(pool), pool.refs)
        for s in range(slots):
            assert pool.lens[s] == len(want[s])
            assert [pool.pages[pool.table[s, i // S], i % S] for i in range(len(want[s]))] == want[s]


def test_reserve_that_lacks_pages_changes_nothing():
    pool = attn_ref.PoolRef(np.array([1, 2, 0], dtype=np.int32),
                            np.array([[0, 1, -1], [1, -1, -1]], dtype=np.int32),
                            np.array([6, 3], dtype=np.int32), 4, np.zeros((3, 4)))
    before = [a.copy() for a in (pool.refs, pool.table, pool.lens)]
    # slot 0 copies page 1 and adds one; slot 1 keeps page 1 and adds one: three, one is free
    assert pool.reserve([0, 1], [9, 5]) == 2
    assert pool.reserve([0], [13]) == -1 and pool.reserve([2], [1]) == -1
    for a, b in zip(before, (pool.refs, pool.table, pool.lens)):
        assert np.array_equal(a, b)
