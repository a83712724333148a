"""The oracle of rotated, scored and drafted tokens against independent statements."""
import numpy as np
import pytest

from oracle import kv8 as O
from kv8_more_tools import tables


@pytest.mark.parametrize("D,R,first,style", [(64, 64, 0, O.HALVES), (64, 32, 32, O.PAIRS),
                                             (128, 16, 8, O.HALVES), (128, 64, 0, O.PAIRS)])
def test_rotation_is_a_complex_product(D, R, first, style):
    rng = np.random.default_rng(1)
    c, s = tables(50, R)
    x = rng.standard_normal((7, 3, D)).astype(np.float32)
    pos = np.array([0, 1, 49, 7, 50, -1, 20])
    y = O.rotate(x, pos, c, s, first, style)
    part = x[..., first:first + R].astype(np.float64)
    z = (part[..., : R // 2] + 1j * part[..., R // 2:] if style == O.HALVES
         else part[..., ::2] + 1j * part[..., 1::2])
    turn = np.ones((7, 1, R // 2), complex)
    ok = (pos >= 0) & (pos < 50)
    turn[ok, 0] = c[pos[ok]].astype(np.float64) + 1j * s[pos[ok]]
    z = z * turn
    want = x.astype(np.float64)
    want[..., first:first + R] = (np.concatenate([z.real, z.imag], -1) if style == O.HALVES
                                  else np.stack([z.real, z.imag], -1).reshape(7, 3, R))
    # two products and a sum, each rounded by half a step of values up to |x0| + |x1|
    size = np.abs(x).max()
    assert np.abs(y - want).max() <= 4 * 2.0 ** -24 * 2 * size
    assert np.array_equal(y[~ok], x[~ok]) and np.array_equal(y[0], x[0])


def test_scored_attention_without_scores_is_attention():
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal(s) for s in ((5, 3, 64), (20, 64), (20, 64)))
    p = 20 - 5 + np.arange(5)
    j = np.arange(20)
    o, lse, a, big = O.attention(q, k, v, 0.125)
    o2, lse2, _, _ = O.attend(q, k, v, 0.125, O.sees(p, j, 20), p[:, None] - j)
    assert np.allclose(o, o2, rtol=0, atol=1e-14) and np.allclose(lse, lse2, rtol=0, atol=1e-13)
    # a cap far above the scores: cap tanh(x / cap) = x - x^3 / (3 cap^2) + ..
    o3, lse3, _, _ = O.attend(q, k, v, 0.125, O.sees(p, j, 20), p[:, None] - j, cap=1e5)
    assert np.allclose(o, o3, rtol=0, atol=1e-8) and np.allclose(lse, lse3, rtol=0, atol=1e-8)


def test_windows_sinks_prefixes():
    j = np.arange(10)
    see = O.sees([-2, 0, 4, 9], j, 10, window=3, sink=2, prefix=0)
    assert [list(np.nonzero(r)[0]) for r in see] == [[], [0], [0, 1, 2, 3, 4], [0, 1, 7, 8, 9]]
    see = O.sees([-2, 0, 4, 9], j, 10, prefix=3)
    assert [int(r.sum()) for r in see] == [3, 3, 5, 10]
    see = O.sees([0, 6], j, 10, window=4, prefix=5)
    assert [list(np.nonzero(r)[0]) for r in see] == [[0, 1, 2, 3, 4], [3, 4, 5, 6]]
    # a window of one leaves each query its own row, whose V comes out
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal(s) for s in ((10, 2, 64), (10, 64), (10, 64)))
    o, lse, _, _ = O.attend(q, k, v, 0.1, O.sees(j, j, 10, window=1), j[:, None] - j)
    assert np.allclose(o, v[:, None], rtol=0, atol=1e-15)
    # a steep slope does the same
    o, _, _, _ = O.attend(q, k, v, 0.1, O.sees(j, j, 10), j[:, None] - j, slopes=[1e4, 1e4])
    assert np.allclose(o, v[:, None], rtol=0, atol=1e-15)


def test_a_tree_that_is_a_chain_is_causal_attention():
    parent = [-1, 0, 1, 2, 3]
    paths = [O.path_to(parent, i) for i in range(5)]
    assert paths[3] == [3, 2, 1, 0]
    assert O.path_to([-1, -1, 0, 7, 2], 4) == [4, 2, 0]
    assert O.path_to([-1, -1, 0, 7, 2], 3) == [3] and O.path_to([0, -5], 0) == [0]


def test_gradient_of_the_cap():
    """cap tanh(x / cap) has slope 1 - tanh^2, against differences of the oracle's lse: with
    one row, lse is the capped score."""
    q = np.array([[[1.0] + [0.0] * 63]])
    for x in (0.0, 3.0, -20.0, 45.0):
        def lse(y):
            k = np.zeros((1, 64))
            k[0, 0] = y
            return O.attend(q, k, k, 1.0, np.ones((1, 1), bool), np.zeros((1, 1)), cap=30.0)[1][0, 0]
        d = (lse(x + 1e-4) - lse(x - 1e-4)) / 2e-4
        assert abs(d - (1 - np.tanh(x / 30.0) ** 2)) < 1e-7
