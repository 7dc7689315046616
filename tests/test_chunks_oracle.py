"""The plain forms of the calls around chunks, pinned by worked examples."""
import math

import numpy as np
import pytest

import _chunks
import _paged
from _paged import BLOCK


def test_rotate_example():
    # a quarter of a turn a position: (a, b) -> (-b, a) -> (-a, -b)
    x = np.arange(1.0, 9.0).reshape(1, 1, 8).repeat(3, 0)
    f = [math.pi / 2, 0.0]
    y, tol = _chunks.rotate(x, None, 0, [0, 1, 2], f, 4, False, 1.0, 0.0)
    np.testing.assert_allclose(y[0, 0], x[0, 0], atol=1e-12)
    np.testing.assert_allclose(y[1, 0], [-3, 2, 1, 4, 5, 6, 7, 8], atol=1e-12)
    np.testing.assert_allclose(y[2, 0], [-1, 2, -3, 4, 5, 6, 7, 8],
                               atol=1e-12)
    y, tol = _chunks.rotate(x, None, 0, [1, 1, 1], f, 4, True, 2.0, 0.0)
    np.testing.assert_allclose(y[0, 0], [-4, 2, 6, 8, 5, 6, 7, 8], atol=1e-12)
    w = np.full(8, 2.0)
    y, tol = _chunks.rotate(np.full((1, 1, 8), 3.0), w, 16.0, [0], [], 0,
                            False, 1.0, 0.0)
    np.testing.assert_allclose(y, 2 * 3 / 5)
    assert (tol < 1e-4).all()


def test_far_angles():
    p, f = 2 ** 31 - 1, 0.7
    assert math.isclose(math.cos(_chunks.turn_of(p, f)),
                        math.cos(math.fmod(p * f, 2 * math.pi)), abs_tol=1e-6)


def test_seen():
    seen = _chunks.seen_by([-1, 0, 4], 6, 1, 2)
    assert seen.tolist() == [[False] * 6, [True] + [False] * 5,
                             [True, False, False, True, True, False]]


@pytest.mark.parametrize("sink,window", [(0, 0), (3, 7)])
def test_chunks_are_single_tokens(sink, window):
    """Each row is the single-token form over the tokens up to it."""
    rng = np.random.default_rng(sink)
    lens, news = [37, 20, 5], [5, 20, 0]
    _, k, v, table, lens = _paged.paged_case(3, lens, 4, 2, 64)
    cu = np.concatenate([[0], np.cumsum(news)])
    q = rng.standard_normal((cu[-1] + 2, 4, 64))
    got = _chunks.attend_chunks(q, k, v, table, cu, lens, sink, window, 0.125,
                                0.0)
    assert got[4].tolist() == [True] * 25 + [False] * 2
    for r in range(3):
        for i in range(news[r]):
            n = lens[r] - news[r] + i + 1
            one = _paged.attend(q[cu[r] + i][None], k, v, table[r][None], [n],
                                sink, window, 0.125, 0.0)
            np.testing.assert_allclose(got[0][cu[r] + i], one[0][0],
                                       rtol=1e-9)
            np.testing.assert_allclose(got[1][cu[r] + i], one[1][0],
                                       rtol=1e-9)


def test_infinite_values_reach_who_attends():
    p = np.array([[0.5, 0.5], [1.0, 0.0]])
    v = np.array([[1.0, 2.0], [np.inf, 4.0]])
    seen = np.array([[True, True], [True, False]])
    o = _chunks.masked_product(p, v, seen)
    assert o.tolist() == [[np.inf, 3.0], [1.0, 2.0]]


def test_weights_of_a_row_sum_to_one():
    lens, news = [40, 17], [3, 17]
    _, k, v, table, lens = _paged.paged_case(5, lens, 4, 2, 64)
    cu = [0, 3, 20]
    q = np.random.default_rng(0).standard_normal((20, 4, 64))
    lse = _chunks.attend_chunks(q, k, v, table, cu, lens, 2, 9, 0.1, 0.0)[1]
    acc = np.ones((2, 64))
    out, tol = _chunks.weigh(q, k, table, cu, lens, 2, 9, 0.1, lse, 0.5, acc)
    np.testing.assert_allclose(out[0, :40].sum(), 3 * 4 + 0.5 * 40)
    np.testing.assert_allclose(out[1, :17].sum(), 17 * 4 + 0.5 * 17)
    assert (out[0, 40:] == 1).all() and (tol < 1e-2).all()


def test_evict_example():
    acc = np.array([[9, 1, 5, 5, 0, 5, 2, 3.]])
    acc = np.pad(acc, ((0, 0), (0, 24)))
    pool = np.arange(3 * BLOCK).reshape(3, BLOCK, 1)
    kept, out, after, pools, bad = _chunks.evict(
        acc, [8], 5, 1, 2, np.array([[1, 0]]), np.array([[2, -1]]), [pool],
        False)
    # the first, the last two, and the first two of the three fives
    assert kept.tolist() == [[0, 2, 3, 6, 7]] and after.tolist() == [5]
    assert out[0, :9].tolist() == [9, 5, 5, 2, 3, 0, 0, 0, 0]
    assert pools[0][2, :6, 0].tolist() == [16, 18, 19, 22, 23, 37]
    assert not bad
