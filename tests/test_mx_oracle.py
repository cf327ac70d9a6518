"""Pins of the microscaled formats', the norm's and sampling's float64 oracle: closed forms, brute
force, invariants."""

import math

import numpy as np
import pytest

from oracle import mx_ref


def test_numbers_of_the_formats():
    assert mx_ref.numbers("fp4").tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    f8 = mx_ref.numbers("fp8")
    assert f8[0] == 0 and f8[1] == 2.0 ** -9 and f8[8] == 2.0 ** -6 and f8[0x38] == 1.0 and f8[-1] == 448
    assert (np.diff(f8) > 0).all() and len(f8) == 127


def test_rounding_to_nearest_even_by_hand():
    # one block, its largest value 4: scale 1 for fp4
    v = [4, 0.25, 0.2501, 0.75, 0.7499, 1.25, 1.75, 2.5, 2.51, 3.5, -0.25, -5.0 / 4]
    want = [4, 0, 0.5, 1, 0.5, 1, 2, 2, 3, 4, 0, -1]
    x = np.zeros((1, 32))
    x[0, :len(v)] = v
    codes, scales = mx_ref.quantize_ref(x, "fp4")
    assert scales.tolist() == [[127]]
    assert mx_ref.values_ref(codes, scales, "fp4")[0, :len(v)].tolist() == want
    # saturation: 7.9 has the scale of 4
    assert mx_ref.held_ref(np.full((1, 1), 7.9), "fp4").tolist() == [[6]]
    assert mx_ref.held_ref(np.full((1, 1), 511.0), "fp8").tolist() == [[448]]
    # halves of a step of 2^-9 (fp8 at scale 1)
    x[0, :5] = [256, 2.0 ** -10, 3 * 2.0 ** -10, 5 * 2.0 ** -10, -2.0 ** -11]
    assert mx_ref.held_ref(x, "fp8")[0, :5].tolist() == [256, 0, 2 * 2.0 ** -9, 2 * 2.0 ** -9, 0]


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_rounding_against_all_numbers(fmt):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 70)) * np.exp(3 * rng.standard_normal((50, 1)))
    codes, scales = mx_ref.quantize_ref(x, fmt)
    held = mx_ref.values_ref(codes, scales, fmt)
    assert scales.shape == (50, 3)
    for r in range(50):
        for c in range(70):
            s = 2.0 ** (int(scales[r, c // 32]) - 127)
            best = np.min(np.abs(np.abs(x[r, c]) - s * mx_ref.numbers(fmt)))
            assert abs(x[r, c] - held[r, c]) == best
    block = np.abs(np.pad(x, ((0, 0), (0, 26)))).reshape(50, 3, 32).max(-1)
    assert (2.0 ** (scales - 127.0 + mx_ref.TOP[fmt]) <= block).all()
    assert (block < 2.0 ** (scales - 127.0 + mx_ref.TOP[fmt] + 1)).all()


def test_ends_of_the_scale():
    x = np.array([[2.0 ** -149] + [0] * 31, [0] * 32, [2.0 ** 127] + [0] * 31, [np.nan] + [1] * 31,
                  [1] * 31 + [-np.inf]])
    _, scales = mx_ref.quantize_ref(x, "fp4")
    assert scales[:, 0].tolist() == [0, 0, 252, 255, 255]
    held = mx_ref.held_ref(x, "fp4")
    assert held[0, 0] == 0 and held[2, 0] == 2.0 ** 127 and np.isnan(held[3:]).all()


def test_tiles_by_hand():
    codes = np.zeros((17, 130), dtype=np.int64)
    codes[3, 70] = 5          # tile 0, block 2, place 6 of row 3: byte 16 (32 + 3) + 3, low half
    codes[16, 129] = 7        # row block 1, tile 1, block 0, place 1 of row 0: high half of byte 0
    scales = np.full((17, 5), 100)
    scales[3, 2] = 33
    t, s = mx_ref.tiled_ref(codes, scales, "fp4")
    assert t.size == 4 * 1024 and t[16 * 35 + 3] == 5 and t[3 * 1024] == 7 << 4 and t.sum() == 5 + (7 << 4)
    assert s.size == 2 * 256 and s[4 * 35] == 33 and s[4 * 35 + 2] == 127 and s[256 + 1] == 100
    t, _ = mx_ref.tiled_ref(codes, scales, "fp8")
    assert t[1024 + 16 * 3 + 6] == 5 and t[3 * 2048 + 1] == 7


def test_norm_closed_forms():
    x = np.array([[3, 4], [0, 0]], dtype=np.float32)
    y, h = mx_ref.norm_ref(x, None, np.array([1, 2], dtype=np.float32), 0.5)
    assert h is x and np.allclose(y, [[3 / math.sqrt(13), 8 / math.sqrt(13)], [0, 0]], rtol=1e-6)
    y, h = mx_ref.norm_ref(x, np.ones_like(x), np.ones(2, dtype=np.float32), 0.0)
    assert h.tolist() == [[4, 5], [1, 1]] and y[1].tolist() == [1, 1]


def test_sampling_closed_forms():
    l = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    for u, token in ((0.0, 1), (0.399, 1), (0.401, 3), (0.699, 3), (0.701, 2), (0.899, 2), (0.901, 0), (2.0, 0)):
        t, lp, n, _ = mx_ref.sample_ref(l, u)
        assert t == token and n == 4 and lp == pytest.approx(l[token])
    assert mx_ref.sample_ref(l, 0.99, top_k=2)[:3] == (3, pytest.approx(math.log(3 / 7)), 2)
    assert mx_ref.sample_ref(l, 0.99, top_p=0.41)[0] == 3 and mx_ref.sample_ref(l, 0.99, top_p=0.39)[0] == 1
    assert mx_ref.sample_ref(l, 0.99, top_p=0.0)[2] == 1
    assert mx_ref.sample_ref(l, 0.99, min_p=0.6)[2] == 2 and mx_ref.sample_ref(l, 0.99, min_p=5.0)[2] == 1
    # p is of what k keeps: 0.4 of 0.7 is over one half
    assert mx_ref.sample_ref(l, 0.99, top_k=2, top_p=0.5)[2] == 1
    assert mx_ref.sample_ref(l, 0.9, temperature=0.0)[:2] == (1, 0.0)
    assert mx_ref.sample_ref(l, 0.9, temperature=float("nan"))[0] == 1
    hot = mx_ref.sample_ref(l, 0.9, temperature=math.inf)
    assert hot[0] == 0 and hot[1] == pytest.approx(math.log(0.25))


def test_sampling_ties_and_what_is_not_finite():
    inf = np.inf
    assert mx_ref.sample_ref(np.zeros(8), 0.3, top_k=4)[:2] == (1, pytest.approx(math.log(0.25)))
    assert mx_ref.sample_ref(np.zeros(8), 0.5, top_p=0.5)[2] == 4
    assert mx_ref.sample_ref(np.array([-inf, np.nan, -inf]), 0.5)[:2] == (-1, -inf)
    assert mx_ref.sample_ref(np.array([1.0, np.nan, -inf]), 0.99)[:2] == (0, 0.0)
    assert mx_ref.sample_ref(np.array([1.0, inf, -inf, inf]), 0.6)[:2] == (3, pytest.approx(math.log(0.5)))


def test_sampling_draws_the_distribution():
    rng = np.random.default_rng(3)
    l = rng.standard_normal(40)
    n = 20000
    hits = np.zeros(40)
    for i in range(n):
        hits[mx_ref.sample_ref(l, (i + 0.5) / n)[0]] += 1
    p = np.exp(l) / np.exp(l).sum()
    assert (np.abs(hits / n - p) <= 1.0 / n).all()
