"""The oracle's rotation and block tables against closed forms and a case worked by hand (no GPU)."""
import numpy as np
import pytest

from oracle import TableOracle, rope_freqs, rope_rows


def test_frequencies():
    assert np.allclose(rope_freqs(8, 10000.0), [1, 0.1, 0.01, 0.001], rtol=1e-15)


@pytest.mark.parametrize("adjacent", [False, True])
def test_quarter_turns(adjacent):
    """At position 1 with a frequency of a quarter turn (a, b) becomes (-b, a); at 2 it changes sign."""
    x = np.arange(1.0, 9.0).reshape(1, 1, 8).repeat(2, 0)
    y, _ = rope_rows(x, [[1, 2]], [np.pi / 2, 0.0], adjacent=adjacent)
    a, b = (0, 1) if adjacent else (0, 2)
    want = x.copy()
    want[0, 0, a], want[0, 0, b] = -x[0, 0, b], x[0, 0, a]
    want[1, 0, [a, b]] *= -1
    assert np.allclose(y, want, atol=1e-14)


def test_products_depend_on_the_distance_only():
    r = np.random.default_rng(0)
    q, k = r.standard_normal((2, 1, 1, 64))
    f = rope_freqs(48, 1e4)
    dot = [float((rope_rows(q, [[p + 7]], f)[0] * rope_rows(k, [[p]], f)[0]).sum()) for p in (0, 5, 4000)]
    assert np.allclose(dot, dot[0], rtol=1e-11)


def test_axes_and_norm():
    r = np.random.default_rng(1)
    x = r.standard_normal((3, 2, 16))
    w = r.standard_normal(16)
    f = rope_freqs(16, 1e3)
    pos = np.array([[5, 0, 9], [0, 7, 9]])
    y, mag = rope_rows(x, pos, f, axes=[0, 1] * 4, weight=w, eps=1e-6)
    n = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-6) * w
    assert np.allclose((y ** 2).sum(-1), (n ** 2).sum(-1))                       # a rotation keeps the length
    assert np.allclose(y[0][:, 1::2], n[0][:, 1::2]) and not np.allclose(y[0][:, 0::2], n[0][:, 0::2])
    assert np.allclose(y[2], rope_rows(n[2:], [[9]], f)[0][0])                  # equal positions: one axis
    assert (mag >= np.abs(y) - 1e-12).all()
    one = rope_rows(x, np.array([[1, 2], [3, 4], [5, 6]]), f)[0]                # a position for every row
    assert np.allclose(one[1, 1], rope_rows(x[1:2], [[4]], f)[0][0, 1])


def test_tables_by_hand():
    t = TableOracle(8, 3, 4)
    assert t.reserve([5, 0, 1]) and t.rows == [[0, 1], [], [2]] and list(t.free) == [3, 4, 5, 6, 7]
    assert t.places([5, 0, 1], [0, 2, 3, 4], 5, [0, 10, 100]) == ([3, 4, -1, 8, -1], [3, 4, 9, 100, 0])
    assert t.reserve([4, 9, 0]) and t.rows == [[0], [3, 4, 5], []] and list(t.free) == [6, 7, 1, 2]
    assert not t.reserve([4, 9, 17]) and t.short == 1 and t.rows == [[0], [3, 4, 5], []]
    assert t.reserve([0, 9, 17]) and t.rows == [[], [3, 4, 5], [6, 7, 1, 2, 0]] and not t.free     # a block given back and taken
