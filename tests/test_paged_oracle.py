"""The plain forms of the paged serving calls, pinned by worked examples."""
import numpy as np

import _paged
from _paged import BLOCK


def test_assign_example():
    table = np.full((3, 2), -1)
    table[1, 0] = 9
    # request 0: new, 17 tokens; 1: grows within its block; 2: into a block
    t, slots, cu, held, head, short = _paged.assign(
        [0, 3, 0], [17, 5, 16], [4, 7, 2, 1], 1, table, 40)
    assert t.tolist() == [[7, 2], [9, -1], [1, -1]]
    assert cu.tolist() == [0, 17, 19, 35]
    assert slots[:19].tolist() == [7 * 16 + i for i in range(16)] + \
        [2 * 16, 9 * 16 + 3, 9 * 16 + 4]
    assert slots[19:35].tolist() == [16 + i for i in range(16)]
    assert (slots[35:] == -1).all()
    assert held.tolist() == [17, 5, 16] and head == 4 and not short


def test_assign_serves_in_order_until_the_list_ends():
    # the second request does not fit, the third would but comes later; the
    # fourth grows inside a block it has
    table = np.array([[-1, -1], [-1, -1], [-1, -1], [5, -1]])
    t, slots, cu, held, head, short = _paged.assign(
        [0, 0, 0, 1], [16, 32, 1, 2], [3, 8], 0, table, 60)
    assert t.tolist() == [[3, -1], [-1, -1], [-1, -1], [5, -1]]
    assert held.tolist() == [16, 0, 0, 2] and head == 1 and short
    assert (slots[16:49] == -1).all() and slots[49] == 5 * BLOCK + 1


def test_attend_example():
    # two tokens with scores 0 and ln 3: weights 1/4 and 3/4
    hd = 64
    q = np.zeros((1, 1, hd)); q[0, 0, 0] = 1.0
    k = np.zeros((2, BLOCK, hd)); v = np.zeros((2, BLOCK, hd))
    k[1, 1, 0] = np.log(3.0)
    v[1, 0, :] = 4.0
    v[1, 1, :] = 8.0
    out, lse, tol, tl = _paged.attend(q, k, v, np.array([[1]]), [2], 0, 0,
                                      1.0, 2.0 ** -8)
    np.testing.assert_allclose(out[0, 0], 7.0, rtol=1e-12)
    np.testing.assert_allclose(lse[0, 0], np.log(4.0), rtol=1e-12)
    assert (tol < 0.05).all() and (tl < 1e-4).all()


def test_attended_positions():
    assert _paged.attended(5, 2, 2).tolist() == [0, 1, 3, 4]
    assert _paged.attended(3, 2, 2).tolist() == [0, 1, 2]
    assert _paged.attended(3, 9, 1).tolist() == [0, 1, 2]
    assert _paged.attended(4, 0, 0).tolist() == [0, 1, 2, 3]
    assert _paged.attended(0, 2, 2).tolist() == []


def test_joining_two_parts_gives_the_whole():
    lens = [40]
    q, k, v, table, lens = _paged.paged_case(3, lens, 2, 1, 64)
    whole = _paged.attend(q, k, v, table, lens, 0, 0, 0.125, 0.0)
    a = _paged.attend(q, k, v, table[:, :1], [16], 0, 0, 0.125, 0.0)
    b = _paged.attend(q, k, v, table[:, 1:], [24], 0, 0, 0.125, 0.0)
    lse = _paged.log_add(a[1], b[1])
    out = (a[0] * np.exp(a[1] - lse)[..., None] +
           b[0] * np.exp(b[1] - lse)[..., None])
    np.testing.assert_allclose(lse, whole[1], rtol=1e-12)
    np.testing.assert_allclose(out, whole[0], rtol=1e-9, atol=1e-12)
