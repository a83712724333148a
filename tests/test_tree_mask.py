"""What drafted tokens see, by the tests' own reckoning (kv8_more_tools.scored_want): against the
oracle's causal attention for a chain, and against masks written out by hand."""
from types import SimpleNamespace

import numpy as np
import pytest

from kv8_more_tools import scored_want
from oracle import kv8 as O

D, G = 8, 2


def held(rng, n):
    """One sequence and head of n rows of small whole numbers, which the codes hold exactly."""
    pair = SimpleNamespace(len=[n], seq={})
    for side in "kv":
        pair.seq[0, 0, side] = s = O.Seq(16, O.INT8, D)
        x = rng.integers(-9, 10, (n, D)).astype(np.float64)
        s.append(x)
        assert np.array_equal(s.values(), x)
    return pair


class Queries(np.ndarray):
    def double(self):
        return self

    def numpy(self):
        return np.asarray(self)


def drafts(rng, T):
    q = rng.standard_normal((1, T, G, D)).view(Queries)
    return q, rng.standard_normal((T, D)), rng.standard_normal((T, D))


@pytest.mark.parametrize("n,T", [(0, 1), (0, 5), (7, 1), (20, 6)])
def test_a_chain_is_causal_attention(n, T):
    rng = np.random.default_rng(1)
    pair, (q, k, v) = held(rng, n), drafts(rng, T)
    o, lse, _, _ = scored_want(pair, q, 0, 0, G, T, 0.3, "f16", k=k, v=v, parent=[i - 1 for i in range(T)])
    rows = [np.concatenate([pair.seq[0, 0, s].values(), x]) for s, x in (("k", k), ("v", v))]
    want, lse2, _, _ = O.attention(np.asarray(q)[0], *rows, 0.3)
    assert np.allclose(o, want, rtol=0, atol=1e-12) and np.allclose(lse, lse2, rtol=0, atol=1e-12)


PARENT = [-1, 0, 0, 1, -1, 3]           # 0 -> 1 -> 3 -> 5, 0 -> 2, and 4 alone
DEPTH = [0, 1, 1, 2, 0, 3]
ALL = [0, 1, 2, 3]                      # cached rows
# (window, first rows): cached rows and drafted tokens that each token sees
MASKS = {
    (0, 0): [(ALL, [0]), (ALL, [0, 1]), (ALL, [0, 2]), (ALL, [0, 1, 3]), (ALL, [4]), (ALL, [0, 1, 3, 5])],
    (3, 0): [([2, 3], [0]), ([3], [0, 1]), ([3], [0, 2]), ([], [0, 1, 3]), ([2, 3], [4]), ([], [1, 3, 5])],
    (3, 2): [(ALL, [0]), ([0, 1, 3], [0, 1]), ([0, 1, 3], [0, 2]), ([0, 1], [0, 1, 3]), (ALL, [4]),
             ([0, 1], [1, 3, 5])],
    (1, 0): [([], [i]) for i in range(6)],
    # first rows that reach into the drafts: the tokens that follow the last row stand at 4
    (1, 5): [(ALL, [0]), (ALL, [0, 1]), (ALL, [0, 2]), (ALL, [0, 3]), (ALL, [4]), (ALL, [0, 5])],
}


@pytest.mark.parametrize("window,sink", MASKS)
@pytest.mark.parametrize("cap", [0.0, 1.5])
@pytest.mark.parametrize("slopes", [None, [0.5, 2.0]])
def test_masks_by_hand(window, sink, cap, slopes):
    rng = np.random.default_rng(2)
    pair, (q, k, v) = held(rng, 4), drafts(rng, 6)
    o, lse, _, _ = scored_want(pair, q, 0, 0, G, 6, 0.1, "f16", cap, window, sink,
                               None if slopes is None else np.array(slopes), k=k, v=v, parent=PARENT)
    kc, vc = (pair.seq[0, 0, s].values() for s in "kv")
    for i, (rows, tokens) in enumerate(MASKS[window, sink]):
        at = [(kc[j], vc[j], j) for j in rows] + [(k[a], v[a], 4 + DEPTH[a]) for a in tokens]
        for g in range(G):
            x = []
            for kk, _, j in at:
                y = 0.1 * float(np.asarray(q)[0, i, g] @ kk)
                y = cap * np.tanh(y / cap) if cap else y
                x.append(y - (slopes[g] * abs(4 + DEPTH[i] - j) if slopes else 0.0))
            w = np.exp(x)
            assert np.allclose(o[i, g], sum(a * vv for a, (_, vv, _) in zip(w, at)) / w.sum(), rtol=0, atol=1e-12)
            assert abs(lse[i, g] - np.log(w.sum())) < 1e-12
