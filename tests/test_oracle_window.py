"""The windowed-attention oracle against closed forms and an independent dense restatement."""
import numpy as np
import pytest

from oracle import window as OW


def test_visible_sets():
    assert OW.visible(9, 10, 0, 0).tolist() == list(range(10))
    assert OW.visible(9, 10, 3, 0).tolist() == [7, 8, 9]
    assert OW.visible(9, 10, 3, 2).tolist() == [0, 1, 7, 8, 9]
    assert OW.visible(9, 10, 3, 8).tolist() == list(range(10))      # sinks reach the window
    assert OW.visible(1, 10, 1, 5).tolist() == [0, 1]               # sinks never show the future
    assert OW.visible(4, 10, 100, 0).tolist() == [0, 1, 2, 3, 4]


def test_rows_that_see_nothing_are_zero():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((5, 64)), rng.standard_normal((2, 64))
    res = OW.prefill(q, k, k, [0, 5], [0, 2], 1, 1, 0, 0, 0.125)    # 5 queries, 2 keys
    for r in range(3):
        assert not res[r][0].any()
    assert np.allclose(res[3][0][0], k[0])                          # position 0 sees itself only


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (7, 3), (64, 0), (5, 40)])
def test_against_dense_softmax(window, sinks):
    rng = np.random.default_rng(window * 10 + sinks)
    nq, nk, Hq, Hkv, d = 9, 23, 4, 2, 64
    q, k, v = (rng.standard_normal((n, h * d)) for n, h in ((nq, Hq), (nk, Hkv), (nk, Hkv)))
    res = OW.prefill(q, k, v, [0, nq], [0, nk], Hq, Hkv, window, sinks, 0.3)
    for hq in range(Hq):
        c = slice((hq // 2) * d, (hq // 2 + 1) * d)
        s = 0.3 * q[:, hq * d:(hq + 1) * d] @ k[:, c].T
        for r in range(nq):
            i = nk - nq + r
            for t in range(nk):
                if t > i or (window and t <= i - window and t >= sinks):
                    s[r, t] = -np.inf
        p = np.exp(s - s.max(1, keepdims=True))
        want = p / p.sum(1, keepdims=True) @ v[:, c]
        got = np.stack([res[r][0][hq] for r in range(nq)])
        assert np.abs(got - want).max() < 1e-12


def test_decode_is_prefill_of_the_newest_row():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 2, 1, 30, 64))          # K and V [B = 2][H = 1][30][64]
    q = rng.standard_normal((2, 128))
    dec = OW.decode(q, k, v, [30, 0], 2, 8, 2, 0.2)
    pre = OW.prefill(q[:1], k[0, 0], v[0, 0], [0, 1], [0, 30], 2, 1, 8, 2, 0.2)
    assert np.allclose(dec[0][0], pre[0][0]) and not dec[1][0].any()
