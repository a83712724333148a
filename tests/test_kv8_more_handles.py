"""Numbers that the C structures of Rope and Scores would change are refused by name."""
import math

import pytest
import torch

import fp4_kv_cache_rope_gb300 as K


@pytest.mark.parametrize("name,value", [
    ("window", 2 ** 32), ("window", 2 ** 32 + 5), ("window", 2 ** 31), ("window", -2 ** 31 - 1), ("sink", 2 ** 32 + 4),
    ("sink", -2 ** 40), ("cap", 1e-46), ("cap", -1e-46), ("cap", 2.0 ** -11), ("cap", 2.0 ** 20 + 1), ("cap", -30.0),
    ("cap", math.inf), ("cap", math.nan), ("cap", 1e39)])
def test_scores(name, value):
    with pytest.raises(K.Csa2Error, match=name):
        K.Scores(**{name: value})


def test_scores_at_the_borders():
    for cap, window, sink in ((0, 2 ** 31 - 1, 2 ** 31 - 1), (2.0 ** -10, 0, 0), (2.0 ** 20, 1, 0), (-0.0, 0, 7)):
        s = K.Scores(cap, window, sink).struct
        assert (s.cap, s.window, s.sink) == (cap, window, sink)


@pytest.mark.parametrize("name,value", [("first", 2 ** 32), ("first", 2 ** 32 + 8), ("style", 2 ** 32 + 1),
                                        ("first", -2 ** 32)])
def test_rope(name, value):
    t = torch.zeros(4, 8)
    with pytest.raises(K.Csa2Error, match=name):
        K.Rope(t, t, **{name: value})
