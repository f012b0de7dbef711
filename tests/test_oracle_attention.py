"""Pins of the attention oracle: closed forms, a brute force in Python, and hand-made page traces (no GPU)."""

import math

import numpy as np

from oracle import attention as oatt


def test_attend_against_a_python_sum():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 4)), rng.standard_normal((5, 4)), rng.standard_normal((5, 4))
    o, lse, a, _ = oatt.attend(q, k, v, 0.5, [0, 1, 2], [5, 4, 2])
    for i, (lo, hi) in enumerate([(0, 5), (1, 4)]):
        w = [math.exp(0.5 * math.fsum(q[i][d] * k[j][d] for d in range(4))) for j in range(lo, hi)]
        total = math.fsum(w)
        for d in range(4):
            assert abs(o[i, d] - math.fsum(x * v[j][d] for x, j in zip(w, range(lo, hi))) / total) < 1e-14
            assert abs(a[i, d] - math.fsum(x * abs(v[j][d]) for x, j in zip(w, range(lo, hi))) / total) < 1e-14
        assert abs(lse[i] - math.log(total)) < 1e-13
    assert (o[2] == 0).all() and np.isneginf(lse[2])


def test_visible_by_hand():
    assert [x.tolist() for x in oatt.visible(3, 3, True, 0)] == [[0, 0, 0], [1, 2, 3]]
    assert [x.tolist() for x in oatt.visible(2, 5, True, 2)] == [[2, 3], [4, 5]]
    assert [x.tolist() for x in oatt.visible(3, 1, True, 0)] == [[0, 0, 0], [0, 0, 1]]
    assert [x.tolist() for x in oatt.visible(2, 4, False, 0)] == [[0, 0], [4, 4]]


def test_prefill_of_equal_scores_is_the_running_mean():
    n, rng = 9, np.random.default_rng(1)
    v = rng.standard_normal((n, 1, 2))
    o, lse, _, _ = oatt.prefill(np.zeros((n, 2, 2)), rng.standard_normal((n, 1, 2)), v, [n], [n], 1.0)
    mean = np.cumsum(v[:, 0], 0) / np.arange(1, n + 1)[:, None]
    assert np.allclose(o[:, 0], mean) and np.allclose(o[:, 1], mean)
    assert np.allclose(lse, np.log(np.arange(1, n + 1))[:, None])


def test_e4m3_round():
    x = [0.0, 1.0, 1.0625, 1.1875, 447.0, 1e9, -500.0, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 464.0]
    y = [0.0, 1.0, 1.0, 1.25, 448.0, 448.0, -448.0, 2.0 ** -9, 0.0, 2.0 ** -8, 448.0]
    assert oatt.e4m3_round(x).tolist() == y
    every = np.array([s * (m / 8 + (e > 0)) * 2.0 ** (max(e, 1) - 7) for s in (1, -1) for e in range(16)
                      for m in range(8) if not (e == 15 and m == 7)])
    assert (oatt.e4m3_round(every) == every).all()


def test_pages_by_hand():
    p = oatt.Pages(6, 4, 4, 3)
    assert p.reserve([0, 1], [5, 4]) == []                       # pages 0, 1 | 2
    assert p.table[:2].tolist() == [[0, 1, -1], [2, -1, -1]] and p.ref.tolist() == [1, 1, 1, 0, 0, 0]
    assert p.fork([0], [2]) == []                                # shares 0, copies 1 to 3
    assert p.table[2].tolist() == [0, 3, -1] and p.content[3] == 1 and p.ref.tolist() == [2, 1, 1, 1, 0, 0]
    p.free([0])
    assert p.ref.tolist() == [1, 0, 1, 1, 0, 0] and p.length[0] == 0
    assert p.reserve([3, 0], [13, 9]) == [0]                     # row 3 wants 4 pages, a table row has 3
    assert p.table[0].tolist() == [1, 4, 5]
    assert p.reserve([1, 2], [1, 1]) == [0]                      # none left for 1; 2 stays inside its page
    p.free([2])
    assert p.compact() == 4                                      # live 1 2 4 5: 4 to 0, 5 to 3
    assert p.table[0].tolist() == [1, 0, 3] and p.ref.tolist() == [1, 1, 1, 1, 0, 0]
    assert p.content[0] == 4 and p.content[3] == 5
